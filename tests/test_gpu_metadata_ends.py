"""GPU: positions and slots at the ends of what their arguments can say: the most tokens a pass can have, and a query_start_loc that
begins past its first token."""
import pytest
import torch

from continuous_batching_paged_ragged_gb300 import pkv

pytestmark = pytest.mark.gpu

MOST = 2**31 - 1


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _equal(got, want):
    """Piece by piece: `want(lo, hi)` makes the values of tokens lo .. hi - 1."""
    for lo in range(0, got.numel(), 1 << 26):
        hi = min(got.numel(), lo + (1 << 26))
        assert torch.equal(got[lo:hi], want(lo, hi)), lo


def test_the_most_tokens(cuda, built):
    pool = pkv.Pool(1, 1, 1, 64, 4)
    ctx, qsl = _i32(MOST), _i32(0, MOST)
    pos = torch.full((MOST,), -1, dtype=torch.int32, device="cuda")
    pkv.pkv_positions(pool.handle, ctx, qsl, 1, MOST, pos)
    _equal(pos, lambda lo, hi: torch.arange(lo, hi, dtype=torch.int32, device="cuda"))
    del pos
    tables = torch.full((1, 1 << 27), 2, dtype=torch.int32, device="cuda")
    slots = torch.full((MOST,), -1, dtype=torch.int64, device="cuda")
    pkv.pkv_slot_mapping(pool.handle, tables, 1 << 27, ctx, qsl, 1, MOST, slots)
    _equal(slots, lambda lo, hi: 32 + (torch.arange(lo, hi, device="cuda") & 15))
    assert pool.check() == 0
    del slots, tables
    torch.cuda.empty_cache()


def test_tokens_in_front_of_the_first_row(cuda, built):
    pool = pkv.Pool(1, 1, 1, 64, 4)
    tables, ctx, qsl = _i32(1, 2).view(1, 2), _i32(3), _i32(5, 8)
    slots = torch.full((8,), 99, dtype=torch.int64, device="cuda")
    pkv.pkv_slot_mapping(pool.handle, tables, 2, ctx, qsl, 1, 8, slots)
    assert slots.tolist() == [-1] * 5 + [16, 17, 18] and pool.check() == pkv.PKV_DEVERR_ROW_META
    pos = torch.full((8,), 99, dtype=torch.int32, device="cuda")
    pkv.pkv_positions(pool.handle, ctx, qsl, 1, 8, pos)
    assert pos.tolist() == [0] * 5 + [0, 1, 2] and pool.check() == pkv.PKV_DEVERR_ROW_META
