"""kda_paged_append with lengths that cross: a token goes to the cache only
where it lies within its sequence's tokens."""
import pytest
import torch

from recompute_kda_chunkwise_gb300 import decode, kda as K

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu", [[0, 9, 1, 1, 9], [0, 4, 2, 3, 9], [0, 3, 3, 9, 9], [0, 9, 9, 2, 9]])
def test_tokens_outside_their_sequence_are_skipped_and_recorded(cu):
    """No row past a sequence's length is written, whatever cu_seqlens holds."""
    N, S, page, lens = 4, 9, 16, [20, 9, 12, 10]
    k = torch.ones(S, 2, 64, dtype=torch.bfloat16, device="cuda")
    kp = torch.zeros(3 * N, page, 2, 64, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.arange(3 * N, **i32).view(N, 3)
    status = torch.zeros(1, **i32)
    decode.paged_append(k, k, kp, vp, table, torch.tensor(lens, **i32), torch.tensor(cu, **i32), status=status)
    written = (kp != 0).any(-1).any(-1).view(N, 3 * page)
    assert torch.equal(kp, vp)
    for n in range(N):
        assert not written[n, lens[n]:].any(), (n, written[n].nonzero().flatten().tolist())
    ordered = all(a <= b for a, b in zip(cu, cu[1:]))
    assert K.query_device_status(status) == (0 if ordered else 6)
    if ordered:
        assert int(written.sum()) == S
