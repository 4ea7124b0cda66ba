"""GPU tests of pa_decode right behind a kernel that writes its lengths and
block table and lets it start early (programmatic dependent launch).

What pa_decode reads before its dependency wait are hints.  The length may
change while its CTAs read it: whichever value each of them sees, the rows have
to be the ones that the same call gives after a synchronisation, bit for bit.
Two writers: the helper of tests/cuda/pdl_writer.cu after a delay that is swept
over the time a decode needs to start, and the library's own
pa_extend_tables."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_pa_gb300 as pa
from gpu_helpers import assert_matches_oracle, ensure_built, to_device
from paged_kv_gqa_pa_gb300 import binding, workloads
from test_pdl_hints_gpu import _slack_pages, writer  # noqa: F401 (a fixture)
from test_q4_gpu import make_decode, to_t

pytestmark = pytest.mark.gpu

KINDS = ["cluster", "merge_kernel", "last_cta", "unsplit", "balanced"]
LENS = [3000, 1200, 2049, 77]


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def make_plan(case, kind):
    """A plan of the kind for the case's shapes (16 query / 4 KV heads, head dim 128)."""
    B, Hq, D = case.q.shape
    S = {"cluster": 256, "merge_kernel": 96, "last_cta": 512, "unsplit": 4096,
         "balanced": binding.PA_PARTITION_BALANCED}[kind]
    plan = pa.pa_plan(B, Hq, case.Hkv, D, 16, case.num_pages, case.max_pages_per_seq,
                      case.max_context_len, case.window, S,
                      torch.cuda.get_device_properties(0).multi_processor_count)
    if kind == "cluster":
        plan.cluster, plan.parts_per_cta, plan.merge_in_kernel = plan.num_partitions, 1, 0
        assert 2 <= plan.num_partitions <= 16
    elif kind in ("merge_kernel", "last_cta"):
        plan.cluster, plan.merge_in_kernel = 0, int(kind == "last_cta")
    assert plan.kernel == 2 and plan.prewait_prefetch > 0
    return plan


class Decode:
    """pa_decode of a case into buffers of its own."""

    def __init__(self, case, kind):
        self.case, self.dev, self.plan = case, to_device(case), make_plan(case, kind)
        B, Hq, D = case.q.shape
        self.out = torch.empty((B, Hq, D), dtype=torch.float16, device="cuda")
        self.lse = torch.empty((B, Hq), dtype=torch.float32, device="cuda")
        self.ws = pa.new_workspace(self.plan, "cuda")

    def __call__(self):
        d = self.dev
        pa.pa_decode(self.plan, d["q"], d["k"], d["v"], d["bt"], d["cl"], self.case.scale,
                     self.case.window, self.out, self.lse, self.ws)

    def rows(self):
        torch.cuda.synchronize()
        assert pa.pa_get_error(self.ws) == 0
        return self.out.clone(), self.lse.clone()


def same(got, want):
    return all(torch.equal(g, w) for g, w in zip(got, want))


# How far the old lengths lie beyond the real ones: with a window of 1000 the first page attended
# moves by 0, 1, 2, 3 and 40 pages.
@pytest.mark.parametrize("window", [0, 1000])
@pytest.mark.parametrize("kind", KINDS)
def test_a_length_that_changes_while_it_is_read(writer, kind, window):  # noqa: F811
    case = workloads.make_case("late", len(LENS), 16, 4, 128, LENS, seed=1700, q_std=2.0,
                               window=window)
    run = Decode(case, kind)
    new_bt, new_cl = run.dev["bt"].clone(), run.dev["cl"].clone()
    run()
    want = run.rows()
    assert_matches_oracle(case, want[0].double().cpu().numpy(), want[1].double().cpu().numpy(),
                          what=f"{kind} window={window}")
    slack = _slack_pages(case)  # (their cells hold NaN)
    old_bt = torch.from_numpy(
        slack[np.arange(case.block_tables.size) % len(slack)].reshape(case.block_tables.shape)).cuda()
    stream = torch.cuda.Stream()
    for moved in (5, 16, 37, 48, 640):
        old_cl = (new_cl + moved).clamp(max=case.max_context_len)
        for delay in range(0, 8001, 250):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                assert writer.launch_delayed_copy(
                    new_bt.data_ptr(), run.dev["bt"].data_ptr(), new_bt.numel(), new_cl.data_ptr(),
                    run.dev["cl"].data_ptr(), new_cl.numel(), delay, stream.cuda_stream) == 0
                run()
            for _ in range(2):
                run.dev["bt"].copy_(old_bt)
                run.dev["cl"].copy_(old_cl)
                graph.replay()
                got = run.rows()
                assert same(got, want), (kind, window, moved, delay)


@pytest.mark.parametrize("window", [0, 1000])
@pytest.mark.parametrize("kind", KINDS)
def test_extend_tables_right_before_pa_decode(kind, window):
    """A graph of the two calls, replayed on requests that are changed in place: a token more, pages
    more, and batch slots that go to other requests."""
    case = workloads.make_case("step", len(LENS), 16, 4, 128, LENS, seed=1701, q_std=2.0,
                               window=window)
    run = Decode(case, kind)
    B, maxp, pages = len(LENS), case.max_pages_per_seq, case.num_pages
    rows = [r[r >= 0] for r in case.block_tables]

    def i32(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")

    # A state: past and new lengths, and which request's pages each batch slot holds.
    states = []
    for lens, new, who in [([2999, 1199, 2048, 76], [1, 1, 1, 1], [0, 1, 2, 3]),
                           ([2999, 1183, 2032, 64], [1, 1, 1, 1], [0, 1, 2, 3]),
                           ([2900, 1150, 2000, 30], [7, 13, 1, 40], [0, 1, 2, 3]),
                           ([76, 2048, 1199, 2999], [1, 1, 1, 1], [3, 2, 1, 0]),
                           ([2048, 76, 0, 1100], [1, 0, 1200, 60], [2, 3, 0, 1])]:
        bt, free = np.full((B, maxp), -1, np.int32), []
        for b in range(B):
            have, need = -(-lens[b] // 16), -(-(lens[b] + new[b]) // 16)
            bt[b, :have] = rows[who[b]][:have]
            free.extend(rows[who[b]][have:need])
        cap = 1300
        states.append((i32(lens), i32(new), i32(free + [0] * (cap - len(free))), i32(bt)))
    past, new, free = (torch.empty_like(x) for x in states[0][:3])
    starts, taken = i32(np.zeros(B + 1)), i32([0])
    slots, pos = torch.zeros(1300, dtype=torch.int64, device="cuda"), i32(np.zeros(1300))
    err = torch.zeros(64, dtype=torch.int32, device="cuda")

    def load(state):
        for dst, src in zip((past, new, free, run.dev["bt"]), state):
            dst.copy_(src)

    def tables():
        pa.pa_extend_tables(past, new, free, pages, run.dev["bt"], run.dev["cl"], starts, slots, pos,
                            taken, err)

    want = []
    for state in states:
        load(state)
        tables()
        torch.cuda.synchronize()
        run()
        want.append(run.rows())
    # (the first state's lengths and pages are the case's own)
    assert_matches_oracle(case, want[0][0].double().cpu().numpy(),
                          want[0][1].double().cpu().numpy(), what=f"{kind} window={window}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tables()
        run()
    order = np.random.default_rng(1).integers(0, len(states), 400)
    for i in order:
        load(states[i])
        graph.replay()
        assert same(run.rows(), want[i]), (kind, window, int(i))
    assert int(err[0]) == 0


@pytest.mark.parametrize("window", [0, 1000])
@pytest.mark.parametrize("lens,cluster", [(LENS, None), (LENS, 0), ([40, 3, 0, 300] * 33, None)])
def test_the_4_bit_decode_behind_a_late_writer(writer, lens, cluster, window):  # noqa: F811
    """The same sweep for pa_q4_decode, whose early start reads lengths and first ids too."""
    q, cache, bt, lens = make_decode(1702, lens, 8, 2, 128, "f16")
    plan = pa.pa_q4_plan(len(lens), 8, 2, 128, 16, cache.shape[0], bt.shape[1], int(lens.max()), window)
    if cluster == 0:
        plan.cluster = 0
    ws, tq = pa.new_workspace(plan, "cuda"), to_t(q, "f16")
    out, lse = torch.empty_like(tq), torch.empty(len(lens), 8, device="cuda")
    new_bt, new_cl = torch.from_numpy(bt).cuda(), torch.from_numpy(lens).cuda()
    now_bt, now_cl = new_bt.clone(), new_cl.clone()

    def run():
        pa.pa_q4_decode(plan, tq, cache, now_bt, now_cl, 0.1, window, out, lse, ws)

    def rows():
        torch.cuda.synchronize()
        assert pa.pa_get_error(ws) == 0
        return out.clone(), lse.clone()

    run()
    want = rows()
    unused = sorted(set(range(cache.shape[0])) - set(bt.ravel().tolist()))  # (NaN scales)
    old_bt = torch.full_like(new_bt, unused[0])
    stream = torch.cuda.Stream()
    for moved in (1, 16, 48, 640):
        old_cl = (new_cl + moved).clamp(max=int(lens.max()))
        for delay in range(0, 8001, 500):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                assert writer.launch_delayed_copy(
                    new_bt.data_ptr(), now_bt.data_ptr(), new_bt.numel(), new_cl.data_ptr(),
                    now_cl.data_ptr(), new_cl.numel(), delay, stream.cuda_stream) == 0
                run()
            for _ in range(2):
                now_bt.copy_(old_bt)
                now_cl.copy_(old_cl)
                graph.replay()
                assert same(rows(), want), (moved, delay)
