"""The paged cache: append and attention against float64 softmax attention.

Bars (tests/_serving_ref.py attention_bar): 2^-8 of sum p |v| for the bf16
probabilities, and the output's own rounding."""
import pytest
import torch

from recompute_kda_chunkwise_gb300 import decode, kda as K
from tests import _serving_ref as R

pytestmark = pytest.mark.gpu


def make(new, lens, Hq, Hkv, D, page, seed=0, std=1.0, spare=3, width=None):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: (torch.randn(*s, generator=g) * std).to(torch.bfloat16).cuda()  # noqa: E731
    need = [-(-max(t, 0) // page) for t in lens]
    pages = sum(need) + spare
    x = {"q": rnd(sum(new), Hq, D), "kp": rnd(pages, page, Hkv, D), "vp": rnd(pages, page, Hkv, D)}
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(new), width or max(max(need), 1)), 2 ** 31 - 1, dtype=torch.int32)  # unused: no page
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    x["table"] = table.cuda()
    x["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    x["cu"] = R.cu_of(new)
    x["cu_t"] = torch.tensor(x["cu"], dtype=torch.int32).cuda()
    return x


def call(x, **kw):
    ws = torch.empty(decode.paged_attention_workspace_bytes(x["q"], x["kp"], x["table"], x["lens"], x["cu_t"]),
                     dtype=torch.uint8).cuda()
    o = decode.paged_attention(x["q"], x["kp"], x["vp"], x["table"], x["lens"], x["cu_t"], workspace=ws, **kw)
    return o, K.query_device_status(ws)


def compare(x, scale=None):
    o, status = call(x, scale=scale)
    assert status == 0
    D = x["q"].shape[2]
    ref, size = R.attention(x["q"], x["kp"], x["vp"], x["table"], x["lens"], x["cu"], D ** -0.5 if scale is None else scale)
    R.check(o, ref, R.attention_bar(size), "o")
    return o


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [8, 16, 24, 64, 128, 256, 200])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (6, 2), (5, 5)])
def test_decode_batches(Hq, Hkv, page, D):
    lens = [1, 2, 127, 128, 129, 255, 256, 300, 511, 1000]
    compare(make([1] * len(lens), lens, Hq, Hkv, D, page, seed=page + D))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,lens", [
    ([1], [1]), ([1], [5000]), ([3, 0, 5, 1], [3, 70, 5, 400]), ([40, 1, 200], [40, 600, 321]), ([130], [130]),
    ([128, 128], [128, 384]), ([300, 17, 0, 64], [300, 1017, 50, 65]), ([129, 127], [700, 127])])
def test_chunks(new, lens, D):
    compare(make(new, lens, 6, 2, D, 16, seed=sum(new)))


@pytest.mark.parametrize("Hq,Hkv", [(128, 1), (160, 1), (3, 1), (96, 8), (7, 7)])
def test_head_layouts(Hq, Hkv):
    compare(make([3, 9], [90, 260], Hq, Hkv, 64, 32, seed=Hq))


def test_many_sequences():
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(1, 200, (700,), generator=g).tolist()
    new = [min(n, int(k)) for n, k in zip(lens, torch.randint(0, 4, (700,), generator=g))]
    compare(make(new, lens, 4, 2, 64, 16, seed=11))


def test_long_sequence_is_split_and_joined():
    compare(make([2], [40000], 8, 2, 128, 64, seed=3))


def test_large_scores_and_a_negative_scale():
    x = make([5, 66], [300, 515], 4, 2, 128, 16, seed=4, std=6.0)
    compare(x)
    compare(x, scale=-0.05)
    compare(x, scale=0.0)


@pytest.mark.parametrize("octaves", [10.0, -10.0, 3.0])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,lens", [([1], [600]), ([140, 2], [600, 333])])
def test_maxima_that_move_all_along_the_keys(new, lens, D, octaves):
    """Scores that rise (or fall) by so many octaves every 32 keys, with noise:
    the running maximum moves inside every tile. The scores stay below 190
    octaves, so three fp32 roundings of them are below 2^-14 of a probability."""
    x = make(new, lens, 2, 1, D, 8, seed=9, std=0.25)
    x["q"][..., 0] = 8.0
    step = octaves / 32 / (8.0 * D ** -0.5 * 1.4426950408889634)
    for n, total in enumerate(lens):
        t = torch.arange(total, device="cuda")
        x["kp"][x["table"][n, t // 8].long(), t % 8, :, 0] = (t * step).to(torch.bfloat16)[:, None]
    compare(x)


def test_rows_that_see_nothing_are_zero():
    """A sequence shorter than its new tokens: the first of them have no position."""
    x = make([6, 4, 150], [2, 0, 20], 4, 2, 64, 16, seed=5)
    o = compare(x)
    assert not o[:4].any() and not o[6:10].any() and not o[10:140].any() and o[140:].any()


@pytest.mark.parametrize("new,lens", [([1, 3, 200], [5, 130, 263])])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf")])
def test_what_lies_past_the_end_is_never_used(new, lens, junk):
    x = make(new, lens, 4, 2, 128, 16, seed=6)
    used = torch.zeros(x["kp"].shape[:2], dtype=torch.bool)
    table = x["table"].cpu()
    for n, t in enumerate(lens):
        for pos in range(t):
            used[int(table[n, pos // 16]), pos % 16] = True
    for p in (x["kp"], x["vp"]):
        p[~used.cuda()] = junk
    compare(x)


def test_nan_in_a_seen_row_stays_with_its_sequence():
    x = make([2, 2], [100, 100], 2, 1, 64, 16, seed=7)
    x["kp"][int(x["table"][0, 0]), 3] = float("nan")
    o, _ = call(x)
    assert torch.isnan(o[:2]).all() and not torch.isnan(o[2:]).any()


def test_append_then_attend():
    new, lens = [3, 0, 40, 1], [3, 9, 100, 65]
    x = make(new, lens, 4, 2, 64, 24, seed=8)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(44, 2, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    kp, vp = x["kp"].clone(), x["vp"].clone()
    status = torch.zeros(1, dtype=torch.int32).cuda()
    decode.paged_append(k, v, x["kp"], x["vp"], x["table"], x["lens"], x["cu_t"], status=status)
    assert K.query_device_status(status) == 0
    for n, t in enumerate(lens):
        for i in range(new[n]):
            pos = t - new[n] + i
            page = int(x["table"][n, pos // 24])
            kp[page, pos % 24], vp[page, pos % 24] = k[x["cu"][n] + i], v[x["cu"][n] + i]
    assert torch.equal(kp, x["kp"]) and torch.equal(vp, x["vp"])
    compare(x)


def test_append_skips_what_does_not_fit():
    x = make([3, 2], [1, 40], 2, 2, 64, 16, seed=9)
    k = torch.ones(5, 2, 64, dtype=torch.bfloat16).cuda()
    kp, vp = x["kp"].clone(), x["vp"].clone()

    def run(**kw):
        y = dict(x, **kw)
        a, b = kp.clone(), vp.clone()
        status = torch.zeros(1, dtype=torch.int32).cuda()
        decode.paged_append(k, k, a, b, y["table"], y["lens"], y["cu_t"], status=status)
        return int((a != kp).any(-1).any(-1).sum()), K.query_device_status(status)

    assert run() == (3, 6)  # two of the first sequence's three tokens have no position
    t = x["table"].clone()
    t[1, 2] = -1
    assert run(table=t) == (1, 6)
    assert run(lens=torch.tensor([3, 49], dtype=torch.int32).cuda()) == (4, 6)  # past the table
    assert run(cu_t=torch.tensor([0, 3, 4], dtype=torch.int32).cuda())[1] == 6


def test_attention_refuses_bad_lengths_and_pages_on_the_device():
    x = make([2, 3], [50, 60], 2, 1, 64, 16, seed=10)
    ref, size = R.attention(x["q"], x["kp"], x["vp"], x["table"], x["lens"], x["cu"], 0.125)
    t = x["table"].clone()
    t[0, 1] = x["kp"].shape[0]
    for bad in ({"table": t}, {"lens": torch.tensor([65, 60], dtype=torch.int32).cuda()},
                {"lens": torch.tensor([-3, 60], dtype=torch.int32).cuda()}):
        o, status = call(dict(x, **bad))
        assert status == 6 and not o[:2].any()
        R.check(o[2:], ref[2:], R.attention_bar(size[2:]), "the other sequence")
    for cu in ([0, 2, 4], [1, 2, 5], [0, 7, 5], [0, -1, 5], [0, 2, 9]):
        _, status = call(dict(x, cu_t=torch.tensor(cu, dtype=torch.int32).cuda()))
        assert status == 6, cu


def test_pages_past_32_bit_offsets():
    """A cache of more than 2^32 elements: the last pages are addressed in 64 bits."""
    page, Hkv, D = 256, 8, 128
    pages = (1 << 32) // (page * Hkv * D) + 4
    small = make([2], [600], 16, Hkv, D, page, seed=12, spare=0)
    kp = torch.empty(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    kp[-3:], vp[-3:] = small["kp"], small["vp"]
    o, status = call(dict(small, kp=kp, vp=vp, table=small["table"] + pages - 3))
    ref, size = R.attention(small["q"], small["kp"], small["vp"], small["table"], small["lens"], small["cu"], D ** -0.5)
    assert status == 0
    R.check(o, ref, R.attention_bar(size), "o")


def test_same_bits_every_run_and_another_stream():
    x = make([2, 70], [3000, 900], 8, 2, 128, 64, seed=13)
    a, _ = call(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = decode.paged_attention(x["q"], x["kp"], x["vp"], x["table"], x["lens"], x["cu_t"])
    s.synchronize()
    assert torch.equal(a, b)
