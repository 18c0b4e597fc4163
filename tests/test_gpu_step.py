"""The recurrent step (kda_step, kda_gdn2_step) against the float64 recurrence.

Bars: every sum is fp32 over at most 128 terms, so outputs and states are held
to the package's fp32 bar, 1e-4 of the RMS, beyond the rounding of the output."""
import pytest
import torch

from recompute_kda_chunkwise_gb300 import decode, kda as K
from tests import _serving_ref as R

pytestmark = pytest.mark.gpu
BAR = 1e-4


def make(lengths, H, D, dtype, gdn2, seed=0, slots=None):
    g = torch.Generator().manual_seed(seed)
    S, slots = sum(lengths), slots or len(lengths) + 2
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g) * std  # noqa: E731
    x = {n: rnd(S, H, D).to(dtype).cuda() for n in ("q", "k", "v", "g")}
    x["gates"] = [rnd(S, H, D).to(dtype).cuda() for _ in range(2)] if gdn2 else [rnd(S, H).to(dtype).cuda()]
    x["A_log"], x["dt_bias"] = rnd(H, std=0.3).cuda(), rnd(H, D, std=0.3).cuda()
    x["states"] = rnd(slots, H, D, D, std=0.5).cuda()
    x["index"] = torch.randperm(slots, generator=g)[: len(lengths)].to(torch.int32).cuda()
    x["cu"] = R.cu_of(lengths)
    x["cu_t"] = torch.tensor(x["cu"], dtype=torch.int32).cuda()
    return x


def call(x, states, commit=None, index="own", **kw):
    f = decode.gdn2_step if len(x["gates"]) == 2 else decode.kda_step
    return f(x["q"], x["k"], x["v"], x["g"], *x["gates"], x["A_log"], x["dt_bias"], x["cu_t"], states,
             state_index=x["index"] if index == "own" else index, commit=commit, **kw)


def ref(x, commit=None, index="own", **kw):
    return R.step(x["q"], x["k"], x["v"], x["g"], x["gates"], x["A_log"], x["dt_bias"], x["cu"], x["states"],
                  x["index"] if index == "own" else index, commit, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gdn2", [False, True])
@pytest.mark.parametrize("lengths", [[1], [1, 1, 1], [0, 5, 1, 4, 0, 9, 3], [37]])
def test_step_matches_recurrence(lengths, gdn2, D, dtype):
    x = make(lengths, 3, D, dtype, gdn2, seed=len(lengths) + D)
    o_ref, pool_ref = ref(x, scale=0.25)
    states = x["states"].clone()
    o = call(x, states, scale=0.25)
    R.check(o, o_ref, BAR, "o")
    R.check(states, pool_ref, BAR, "states")


@pytest.mark.parametrize("gdn2", [False, True])
def test_commit_keeps_the_state_after_the_committed_tokens(gdn2):
    lengths = [6, 5, 4, 1, 0, 8, 2]
    x = make(lengths, 2, 128, torch.bfloat16, gdn2, seed=4)
    commit = torch.tensor([0, 5, 2, 1, 0, 7, 99], dtype=torch.int32).cuda()  # 99: more than there are
    o_ref, pool_ref = ref(x, commit=commit)
    states = x["states"].clone()
    o = call(x, states, commit=commit)
    R.check(o, o_ref, BAR, "o")
    R.check(states, pool_ref, BAR, "states")
    untouched = [s for s in range(states.shape[0]) if s not in x["index"].tolist()] + [int(x["index"][0]), int(x["index"][4])]
    for s in untouched:
        assert torch.equal(states[s], x["states"][s])


def test_default_slots_inactive_sequences_and_an_output_buffer():
    x = make([2, 3, 1], 2, 64, torch.float32, False, seed=9)
    o_ref, pool_ref = ref(x, index=None)
    states = x["states"].clone()
    out = torch.full_like(x["q"], float("nan"))
    assert call(x, states, index=None, out=out) is out
    R.check(out, o_ref, BAR, "o")
    R.check(states, pool_ref, BAR, "states")
    index = torch.tensor([3, -1, 0], dtype=torch.int32).cuda()
    o_ref, pool_ref = ref(x, index=index)
    states = x["states"].clone()
    o = call(x, states, index=index, out=torch.full_like(x["q"], float("nan")))
    R.check(o, o_ref, BAR, "o with an inactive sequence")
    R.check(states, pool_ref, BAR, "states with an inactive sequence")


def test_tokens_split_over_calls_are_bit_identical():
    x = make([7, 7], 2, 128, torch.bfloat16, False, seed=2)
    whole = x["states"].clone()
    o = call(x, whole)
    parts = x["states"].clone()
    for lo, hi in ((0, 3), (3, 4), (4, 7)):
        rows = torch.cat([torch.arange(lo, hi), torch.arange(7 + lo, 7 + hi)]).cuda()
        y = {k: (x[k][rows].contiguous() if k in "qkvg" else x[k]) for k in x}
        y["gates"] = [t[rows].contiguous() for t in x["gates"]]
        y["cu_t"] = torch.tensor([0, hi - lo, 2 * (hi - lo)], dtype=torch.int32).cuda()
        assert torch.equal(call(y, parts), o[rows])
    assert torch.equal(parts, whole)


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_continues_a_chunked_prefill(dtype, D):
    """Prefill with kda_fwd, then decode with kda_step: the outputs and the
    state of the whole sequence in one recurrence."""
    x = make([100, 33], 2, D, dtype, False, seed=6, slots=2)
    x["index"] = torch.tensor([0, 1], dtype=torch.int32).cuda()
    x["states"].zero_()
    o_ref, pool_ref = ref(x)
    cut = [90, 20]
    head = torch.cat([torch.arange(0, 90), torch.arange(100, 120)]).cuda()
    tail = torch.cat([torch.arange(90, 100), torch.arange(120, 133)]).cuda()
    part = lambda rows: [x[n][rows].contiguous() for n in ("q", "k", "v", "g")] + [x["gates"][0][rows].contiguous()]  # noqa: E731
    _, _, hT = K.kda_fwd(*part(head), x["A_log"], x["dt_bias"], torch.tensor(R.cu_of(cut), dtype=torch.int32).cuda(),
                         save_ctx=False, final_state=True)
    o = decode.kda_step(*part(tail), x["A_log"], x["dt_bias"], torch.tensor([0, 10, 23], dtype=torch.int32).cuda(), hT)
    bar = 2e-2 if dtype == torch.bfloat16 else BAR  # the prefill's own bar
    R.check(o, o_ref[tail.cpu()], bar, "o")
    R.check(hT, pool_ref, bar, "states")


def test_extreme_gates_and_zero_vectors():
    x = make([4, 4], 2, 64, torch.float32, False, seed=8)
    x["g"][:2] = 1e4     # decay at the bound
    x["g"][2:4] = -1e4   # no decay
    x["gates"][0][1] = -1e4
    x["gates"][0][2] = 1e4
    x["k"][3] = 0
    x["q"][0] = 0
    o_ref, pool_ref = ref(x)
    states = x["states"].clone()
    o = call(x, states)
    R.check(o, o_ref, BAR, "o")
    R.check(states, pool_ref, BAR, "states")
    assert not o[0].any()


def test_slots_past_32_bit_offsets():
    """A pool of more than 2^31 elements: the last slots are addressed in 64 bits."""
    H, D = 16, 128
    slots = (1 << 31) // (H * D * D) + 3
    x = make([2, 1], H, D, torch.bfloat16, False, seed=3, slots=4)
    pool = torch.zeros(slots, H, D, D, device="cuda")
    pool[slots - 2:] = x["states"][:2]
    o = call(x, pool, index=torch.tensor([slots - 1, slots - 2], dtype=torch.int32).cuda())
    o_ref, pool_ref = ref(x, index=torch.tensor([1, 0]))
    R.check(o, o_ref, BAR, "o")
    R.check(pool[slots - 2:], pool_ref[:2], BAR, "states")
    assert not pool[: slots - 2].any()


def test_device_checks_record_and_skip():
    x = make([2, 2, 2], 2, 64, torch.float32, False, seed=1)
    o_ref, pool_ref = ref(x)
    slots = x["states"].shape[0]

    def run(**kw):
        status = torch.zeros(1, dtype=torch.int32).cuda()
        states = x["states"].clone()
        o = call(dict(x, **kw.pop("x", {})), states, status=status, out=torch.full_like(x["q"], 7.0), **kw)
        return o, states, K.query_device_status(status)

    o, states, st = run()
    assert st == 0
    bad = x["index"].clone()
    bad[1] = slots
    o, states, st = run(index=bad)
    assert st == 6 and bool((o[2:4] == 7).all()) and torch.equal(states[x["index"][1].long()], x["states"][x["index"][1].long()])
    R.check(o[4:], o_ref[4:], BAR, "the other sequences")
    o, states, st = run(commit=torch.tensor([2, -1, 2], dtype=torch.int32).cuda())
    assert st == 6 and bool((o[2:4] == 7).all())
    for cu in ([0, 5, 4, 6], [0, 2, 4, 5], [1, 2, 4, 6], [0, 2, 9, 6], [0, -2, 4, 6]):
        o, states, st = run(x={"cu_t": torch.tensor(cu, dtype=torch.int32).cuda()})
        assert st == 6, cu


def test_on_another_stream():
    x = make([1] * 5, 4, 128, torch.bfloat16, False, seed=5)
    o_ref, pool_ref = ref(x)
    states = x["states"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o = call(x, states)
    s.synchronize()
    R.check(o, o_ref, BAR, "o")
    R.check(states, pool_ref, BAR, "states")
