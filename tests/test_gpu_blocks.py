"""GPU: pkv_copy_blocks, pkv_fork_rows and pkv_compact against numpy on copies of the pool, every byte of it (the calls
move bits, so everything is compared exactly; what no call may touch holds random bytes)."""
import numpy as np
import pytest
import torch

from continuous_batching_paged_ragged_gb300 import pkv

pytestmark = pytest.mark.gpu

KINDS = [pkv.PKV_KV_F16, pkv.PKV_KV_E4M3]
SHAPES = [(1, 1, 64), (3, 2, 128), (2, 4, 256), (28, 2, 128)]  # layers, KV heads, head_dim


class Host:
    """The pool's bytes on the host, as [plane][block][head][slot][row bytes] and scale records."""

    def __init__(self, pool):
        c = pool.cfg
        self.values = pool.cache_view().view(torch.uint8).reshape(2 * c.num_layers, c.num_blocks, c.num_kv_heads, 16, -1).cpu().numpy().copy()
        self.scales = pool.scales_view().cpu().numpy().copy() if pool.is_8bit else None

    def copy(self, src, dst, rows=16):
        self.values[:, dst, :, :rows] = self.values[:, src, :, :rows]
        if self.scales is not None:
            self.scales[:, dst, :, :, :rows] = self.scales[:, src, :, :, :rows]

    def same(self, other):
        assert np.array_equal(self.values, other.values)
        assert self.scales is None or np.array_equal(self.scales, other.scales)


def _pool(layers, hkv, d, blocks, kv, seed=0):
    pool = pkv.Pool(layers, hkv, hkv, d, blocks, kv_dtype=kv)
    pool.buffer[:-256].random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(seed))
    return pool


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("layers,hkv,d", SHAPES)
@pytest.mark.parametrize("n", [1, 7, 150])
def test_copy(cuda, built, kv, layers, hkv, d, n):
    pool = _pool(layers, hkv, d, 2 * n + 3, kv)
    ids = np.random.default_rng(n).permutation(2 * n + 3)
    pairs = np.stack([ids[:n], ids[n:2 * n]], 1)
    pairs[-1, 0] = pairs[0, 0]  # one source, two destinations
    pairs = np.concatenate([pairs, [[-1, 5], [5, -1], [-1, -1]]])
    want = Host(pool)
    for s, t in pairs[:n]:
        want.copy(s, t)
    pkv.pkv_copy_blocks(pool.handle, _dev(pairs), n + 3)
    assert pool.check() == 0
    Host(pool).same(want)


def test_copy_reports_and_skips_bad_ids(cuda, built, monkeypatch):
    pool = _pool(2, 2, 64, 9, pkv.PKV_KV_E4M3)
    want = Host(pool)
    want.copy(3, 4)
    bad = _dev([[0, 9], [-2, 1], [3, 4], [2**30, 2]])
    pkv.pkv_copy_blocks(pool.handle, bad, 4)
    assert pool.check() == pkv.PKV_DEVERR_BLOCK_RANGE
    Host(pool).same(want)
    pkv.pkv_copy_blocks(pool.handle, bad, 0)
    assert pkv.pkv_last_launch_count(pool.handle) == 0
    for args in [(bad, -1), (None, 2)]:
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_copy_blocks(pool.handle, *args)
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG
    monkeypatch.setenv("PKV_VALIDATE", "1")
    for pairs, status in [([[0, 9]], pkv.PKV_ERR_OUT_OF_RANGE), ([[0, 1], [2, 1]], pkv.PKV_ERR_INVALID_ARG),
                          ([[0, 1], [1, 2]], pkv.PKV_ERR_INVALID_ARG), ([[1, 2], [0, 1]], pkv.PKV_ERR_INVALID_ARG),
                          ([[3, 3]], pkv.PKV_ERR_INVALID_ARG)]:
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_copy_blocks(pool.handle, _dev(pairs), len(pairs))
        assert e.value.status == status, pairs
    Host(pool).same(want)
    pkv.pkv_copy_blocks(pool.handle, _dev([[0, 1], [0, 2], [-1, 1]]), 3)


def _fork_host(host, tables, ctx, forks):
    tables, ctx = tables.copy(), ctx.copy()
    for p, c, b in forks:
        full, tail = divmod(int(ctx[p]), 16)
        row = np.full(tables.shape[1], -1, np.int32)
        row[:full] = tables[p, :full]
        if tail:
            row[full] = b
            host.copy(tables[p, full], b, tail)
        tables[c], ctx[c] = row, ctx[p]
    return tables, ctx


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("layers,hkv,d", SHAPES)
@pytest.mark.parametrize("parents,children", [(1, 1), (3, 2), (40, 3)])
def test_fork(cuda, built, kv, layers, hkv, d, parents, children):
    rng = np.random.default_rng(parents)
    ctx = rng.integers(1, 90, parents).astype(np.int32)
    ctx[0] = 15
    if parents > 2:
        ctx[1], ctx[2] = 32, 96  # whole blocks: nothing copied; a full table
    width = 6
    rows = parents * (1 + children)
    need = int(sum(-(-c // 16) for c in ctx))
    ids = rng.permutation(need + rows)
    tables = np.full((rows, width), -7, np.int32)  # children's rows hold anything
    at = 0
    for p in range(parents):
        n = -(-int(ctx[p]) // 16)
        tables[p, :n], at = ids[at:at + n], at + n
    lens = np.concatenate([ctx, np.full(rows - parents, 12345, np.int32)])
    forks = [(p, parents + p * children + j, int(ids[need + p * children + j]) if ctx[p] % 16 else -1)
             for p in range(parents) for j in range(children)]
    rng.shuffle(forks)
    pool = _pool(layers, hkv, d, need + rows, kv)
    want = Host(pool)
    wt, wc = _fork_host(want, tables, lens, forks)
    dt, dc = _dev(tables), _dev(lens)
    pkv.pkv_fork_rows(pool.handle, dt, width, dc, rows, _dev(forks + [(-1, 0, 0)]), len(forks) + 1)
    assert pool.check() == 0
    assert np.array_equal(dt.cpu().numpy(), wt) and np.array_equal(dc.cpu().numpy(), wc)
    Host(pool).same(want)


def test_fork_reports_and_skips_bad_forks(cuda, built, monkeypatch):
    pool = _pool(2, 2, 128, 10, pkv.PKV_KV_F16)
    tables = np.array([[0, 1], [2, 99], [-1, -1], [3, 4], [5, -1], [6, 6]], np.int32)
    ctx = np.array([20, 30, -5, 33, 0, 16], np.int32)
    cases = [((0, 6, 7), pkv.PKV_DEVERR_ROW_META), ((6, 1, 7), pkv.PKV_DEVERR_ROW_META), ((-2, 1, 7), pkv.PKV_DEVERR_ROW_META),
             ((0, 0, 7), pkv.PKV_DEVERR_ROW_META), ((2, 4, 7), pkv.PKV_DEVERR_ROW_META), ((3, 4, 7), pkv.PKV_DEVERR_ROW_META),
             ((0, 4, 10), pkv.PKV_DEVERR_BLOCK_RANGE), ((0, 4, -1), pkv.PKV_DEVERR_BLOCK_RANGE),
             ((1, 4, 7), pkv.PKV_DEVERR_BLOCK_RANGE), ((4, 2, -1), 0), ((5, 2, -1), 0)]
    for fork, bits in cases:
        want = Host(pool)
        wt, wc = (tables, ctx) if bits else _fork_host(want, tables, ctx, [fork])
        dt, dc = _dev(tables), _dev(ctx)
        pkv.pkv_fork_rows(pool.handle, dt, 2, dc, 6, _dev([fork]), 1)
        assert pool.check() == bits, fork
        assert np.array_equal(dt.cpu().numpy(), wt) and np.array_equal(dc.cpu().numpy(), wc), fork
        Host(pool).same(want)
    dt, dc = _dev(tables), _dev(ctx)
    for args in [(dt, 0, dc, 6, dt, 1), (None, 2, dc, 6, dt, 1), (dt, 2, None, 6, dt, 1), (dt, 2, dc, -1, dt, 1), (dt, 2, dc, 6, dt, -1),
                 (dt, 2, dc, 6, None, 1)]:
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_fork_rows(pool.handle, *args)
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG
    monkeypatch.setenv("PKV_VALIDATE", "1")
    for forks in [[(0, 1, 7), (3, 1, 8)], [(0, 1, 7), (3, 2, 7)], [(0, 1, 7), (1, 2, 8)], [(0, 9, 7)]]:
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_fork_rows(pool.handle, dt, 2, dc, 6, _dev(forks), len(forks))
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG and "PKV_VALIDATE" in str(e.value)
    assert np.array_equal(dt.cpu().numpy(), tables)


def _compact_host(host, tables, blocks):
    held = sorted({int(x) for x in tables.ravel() if 0 <= x < blocks})
    n = len(held)
    remap = np.full(blocks, -1, np.int32)
    remap[held] = held
    holes = [x for x in range(n) if remap[x] < 0]
    for s, t in zip([x for x in held if x >= n], holes):
        host.copy(s, t)
        remap[s] = t
    new = np.array([[remap[x] if 0 <= x < blocks else x for x in row] for row in tables], np.int32).reshape(tables.shape)
    return new, remap, n


def _compact(pool, tables, in_place=False):
    dt = _dev(tables)
    new = dt if in_place else torch.full_like(dt, -9)
    remap, live = torch.full((pool.cfg.num_blocks,), -9, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    n = pkv.pkv_compact_workspace_bytes(pool.handle)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    pkv.pkv_compact(pool.handle, dt, tables.shape[1], tables.shape[0], new, remap, live, ws, n)
    return new.cpu().numpy(), remap.cpu().numpy(), int(live)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("layers,hkv,d", SHAPES)
@pytest.mark.parametrize("blocks,rows,width,used", [(1, 1, 1, 1), (33, 2, 5, 8), (64, 4, 20, 64), (500, 7, 30, 120), (700, 20, 40, 690),
                                                    (2048, 32, 32, 700), (2049, 8, 16, 100), (600, 33, 32, 300)])
def test_compact(cuda, built, kv, layers, hkv, d, blocks, rows, width, used):
    rng = np.random.default_rng(blocks + used)
    tables = np.full((rows, width), -1, np.int32)
    places = rng.permutation(rows * width)
    ids = rng.permutation(blocks)[:used]
    tables.ravel()[places[:min(used, rows * width)]] = ids[:rows * width]
    if used + 5 < rows * width:
        tables.ravel()[places[used:used + 5]] = ids[0]  # a shared block
    pool = _pool(layers, hkv, d, blocks, kv)
    want = Host(pool)
    wt, wr, wn = _compact_host(want, tables, blocks)
    for in_place in (False, True):
        p = _pool(layers, hkv, d, blocks, kv)
        new, remap, n = _compact(p, tables, in_place)
        assert n == wn and np.array_equal(new, wt) and np.array_equal(remap, wr)
        Host(p).same(want)
        assert p.check() == 0


@pytest.mark.parametrize("blocks,rows,width", [(420000, 4, 100), (3000, 300, 300), (3000, 128, 128), (3000, 129, 127)])
def test_compact_large_pools_and_tables(cuda, built, blocks, rows, width):
    """The bitmap in the workspace: a pool past 48 KB of bits, and tables past 16 K entries (and at them)."""
    rng = np.random.default_rng(1)
    tables = rng.integers(-1, blocks, (rows, width)).astype(np.int32)
    tables[0, 0], tables[1, 1], tables[2, 2] = blocks - 1, 0, -1
    pool = _pool(1, 1, 64, blocks, pkv.PKV_KV_E4M3)
    want = Host(pool)
    wt, wr, wn = _compact_host(want, tables, blocks)
    new, remap, n = _compact(pool, tables)
    assert n == wn and np.array_equal(new, wt) and np.array_equal(remap, wr) and pool.check() == 0
    Host(pool).same(want)


@pytest.mark.parametrize("blocks", [385024, 385025, 393100, 393216, 393217])
def test_compact_pools_whose_bitmap_about_fills_shared_memory(cuda, built, blocks):
    rng = np.random.default_rng(blocks)
    tables = rng.integers(-1, blocks, (40, 60)).astype(np.int32)
    tables[0, 0], tables[1, 1] = blocks - 1, 0
    pool = _pool(1, 1, 64, blocks, pkv.PKV_KV_E4M3)
    want = Host(pool)
    wt, wr, wn = _compact_host(want, tables, blocks)
    new, remap, n = _compact(pool, tables)
    assert n == wn and np.array_equal(new, wt) and np.array_equal(remap, wr) and pool.check() == 0
    Host(pool).same(want)


def test_compact_edges_and_refusals(cuda, built):
    pool = _pool(1, 2, 64, 40, pkv.PKV_KV_F16)
    want = Host(pool)
    # nothing in use; then ids that name no block
    new, remap, n = _compact(pool, np.full((3, 4), -1, np.int32))
    assert n == 0 and (new == -1).all() and (remap == -1).all() and pool.check() == 0
    tables = np.array([[39, 40, -2], [7, -1, 2**31 - 1]], np.int32)
    wt, wr, wn = _compact_host(want, tables, 40)
    new, remap, n = _compact(pool, tables)
    assert n == 2 and np.array_equal(new, wt) and np.array_equal(remap, wr) and pool.check() == pkv.PKV_DEVERR_BLOCK_RANGE
    Host(pool).same(want)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    nb = pkv.pkv_compact_workspace_bytes(pool.handle)
    t, r, l, ws = i32(2, 3), i32(40), i32(1), torch.empty(nb + 256, dtype=torch.uint8, device="cuda")
    pkv.pkv_compact(pool.handle, None, 1, 0, None, r, l, ws, nb)  # no rows: every block is free
    assert int(l) == 0 and (r == -1).all()
    for args in [(t, 0, 2, t, r, l, ws, nb), (t, 3, -1, t, r, l, ws, nb), (None, 3, 2, t, r, l, ws, nb), (t, 3, 2, None, r, l, ws, nb),
                 (t, 3, 2, t, None, l, ws, nb), (t, 3, 2, t, r, None, ws, nb), (t, 3, 2, t, r, l, None, nb), (t, 3, 2, t, r, l, ws, nb - 1),
                 (t, 3, 2, t, r, l, ws.data_ptr() + 16, nb)]:
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_compact(pool.handle, *args)
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG
        assert pkv.pkv_last_launch_count(pool.handle) == 0
