"""gemm_lora and gemm_lora_backward on the GPU against tests/rows_reference.py (NumPy,
float64): within bounds derived beside them, and bit for bit where every sum is exact.

Inputs lie inside NaN-filled buffers (rows' padding, ranks that an adapter does not have,
adapters that no row has), outputs inside ones filled with a sentinel that has to survive."""
import numpy as np
import pytest

import mx_reference as mxref
import rows_reference as ref
from fp32_gemm_07_amd import binding as lib
from gpu_util import say, torch

pytestmark = pytest.mark.gpu

KINDS = {"f32": 0, "bf16": 1, "f16": 2}
SENTINEL = -77.0


@pytest.fixture(scope="module", autouse=True)
def _setup():
    lib.load()
    torch()


def dtype(kind):
    t = torch()
    return {"f32": t.float32, "bf16": t.bfloat16, "f16": t.float16}[kind]


def stream():
    return torch().cuda.current_stream().cuda_stream


def dev(x, kind="f32"):
    return torch().from_numpy(np.ascontiguousarray(x, np.float32)).to("cuda:0").to(dtype(kind))


def dev_ints(x):
    return None if x is None else torch().from_numpy(np.ascontiguousarray(x, np.int32)).to("cuda:0")


def host(x):
    return x.float().cpu().numpy()


def padded(x, kind, pad, offset=0, fill=np.nan):
    rows, cols = x.shape
    buf = np.full(offset + rows * (cols + pad) + 8, fill, np.float32)
    buf[offset:offset + rows * (cols + pad)].reshape(rows, cols + pad)[:, :cols] = x
    return dev(buf, kind)[offset:], cols + pad


class Case:
    """Inputs of one call, already rounded to their type."""

    def __init__(self, rng, rows, n, k, rank, adapters, kind, mixed, whole=False, pad=0, offset=0):
        self.rows, self.n, self.k, self.rank, self.adapters, self.kind, self.pad, self.offset = rows, n, k, rank, adapters, kind, pad, offset

        def values(*shape, spread=1.0):
            if whole:   # small whole numbers: every sum is exact
                return rng.integers(-2, 3, shape).astype(np.float32)
            return mxref.to_type((rng.normal(size=shape) * spread).astype(np.float32), KINDS[kind])

        self.x, self.c, self.dy, self.dc = values(rows, k), values(rows, n), values(rows, n), values(rows, k)
        self.a, self.b = values(adapters, rank, k, spread=k ** -0.5), values(adapters, n, rank, spread=rank ** -0.5)
        self.ids = rng.integers(0, adapters, rows).astype(np.int32)
        if not mixed:
            self.ids = np.sort(self.ids)
        if rows > 3:
            self.ids[rng.integers(0, rows, rows // 8)] = rng.choice([-1, adapters, 2 ** 31 - 1, -2 ** 31])
            if not mixed:
                self.ids[rows - rows // 8:] = -1
        self.ranks = rng.integers(0 if adapters > 1 else 1, rank + 1, adapters).astype(np.int32)
        self.ranks[rng.integers(0, adapters)] = rank
        self.scales = rng.choice([0.5, 1.0, 2.0, -1.0], adapters).astype(np.float32) if whole else rng.normal(size=adapters).astype(np.float32)
        for i in range(adapters):   # what no row uses
            self.a[i, self.ranks[i]:] = np.nan
            self.b[i, :, self.ranks[i]:] = np.nan
            if i not in self.ids:
                self.a[i] = self.b[i] = np.nan

    def set(self, ranks=True, scales=True):
        self.da, self.db = dev(self.a, self.kind), dev(self.b, self.kind)
        self.dr, self.ds, self.di = dev_ints(self.ranks), dev(self.scales), dev_ints(self.ids)
        return lib.gemm_lora_t(KINDS[self.kind], self.n, self.k, self.rank, self.adapters, self.da, self.db, self.dr if ranks else None,
                               self.ds if scales else None)


def run_forward(c, base="other", workspace=True, s=None):
    """Y NumPy; base: "other" buffer, in "place", "none"."""
    t = torch()
    s = s or c.set()
    x, ldx = padded(c.x, c.kind, c.pad, c.offset)
    cd, ldc = padded(c.c, c.kind, c.pad + 1, c.offset, SENTINEL if base == "place" else np.nan)
    if base == "place":
        y, ldy = cd, ldc
    else:
        ldy = c.n + c.pad
        y = t.full((c.rows * ldy + 8,), SENTINEL, device="cuda:0").to(dtype(c.kind))
    need = lib.gemm_lora_workspace_bytes(c.rows, s)
    ws = t.full((need + 16,), 0xff, dtype=t.uint8, device="cuda:0") if workspace else None   # NaN everywhere
    lib.gemm_lora(c.rows, s, c.di, x, ldx, None if base == "none" else cd, ldc, y, ldy, ws, need if workspace else 0, stream())
    out = host(y)
    assert (out[c.rows * ldy:] == SENTINEL).all() or base == "place"
    out = out[:c.rows * ldy].reshape(c.rows, ldy)
    assert (out[:, c.n:] == SENTINEL).all()
    if workspace:
        assert (ws[need:] == 0xff).all()
    return out[:, :c.n]


def half_step(kind, y):
    k = KINDS[kind]
    return np.abs(y) * mxref.HALF_STEP[k] + (2.0 ** -25 if k == 2 else 0)


def check_forward(c, what, base="other", workspace=True, exact=False, **set_args):
    say(what)
    got = run_forward(c, base, workspace, c.set(**set_args) if set_args else None)
    ranks = c.ranks if set_args.get("ranks", True) else None
    scales = c.scales if set_args.get("scales", True) else None
    y, mag = ref.lora(c.x.astype(np.float64), None if base == "none" else c.c, c.a.astype(np.float64), c.b.astype(np.float64), c.ids, ranks, scales)
    if exact:
        assert np.array_equal(got, mxref.to_type(y, KINDS[c.kind])), what
        return
    # K + rank x (up to 5 products of parts) FP32 additions, each off by at most 2^-23 of the magnitudes
    # (a matrix instruction may cut off instead of rounding), as many more where ranges are joined
    # as there are ranges and waves; scale and parts 2^-24 each
    bound = mag * (c.k + 5 * c.rank + 40) * 2.0 ** -23
    bound = bound + half_step(c.kind, np.abs(y) + bound)
    assert (np.abs(got - y) <= bound).all(), (what, np.nanmax(np.abs(got - y) / bound), np.isnan(got).sum())
    none = (c.ids < 0) | (c.ids >= c.adapters)
    assert np.array_equal(got[none], np.zeros_like(c.c[none]) if base == "none" else c.c[none])


SIZES = [  # rows, n, k, rank, adapters
    (1, 1, 1, 1, 1), (1, 64, 64, 16, 3), (1, 4096, 2048, 16, 2), (5, 33, 17, 3, 2), (16, 100, 130, 8, 4), (17, 257, 65, 9, 17), (40, 96, 200, 33, 5),
    (64, 300, 512, 64, 64), (130, 1000, 72, 100, 3), (33, 65, 1030, 128, 2), (300, 513, 777, 24, 6), (2000, 130, 140, 5, 3), (513, 700, 520, 80, 1),
    (20, 2050, 4100, 4, 9)]


@pytest.mark.parametrize("rows,n,k,rank,adapters", SIZES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("mixed", [False, True])
def test_forward(rows, n, k, rank, adapters, kind, mixed):
    rng = np.random.default_rng(rows + n + k + rank)
    c = Case(rng, rows, n, k, rank, adapters, kind, mixed, pad=rows % 3, offset=n % 2)
    for base in ("other", "place", "none"):
        check_forward(c, f"lora {rows}x{n}x{k} r{rank} of {adapters} {kind} mixed {mixed} {base}", base, workspace=base != "none")


@pytest.mark.parametrize("rows,n,k,rank,adapters", SIZES)
@pytest.mark.parametrize("kind", KINDS)
def test_forward_whole_numbers(rows, n, k, rank, adapters, kind):
    rng = np.random.default_rng(rows * 7 + n)
    c = Case(rng, rows, n, min(k, 400), rank, adapters, kind, True, whole=True, pad=1)
    check_forward(c, f"lora whole numbers {rows}x{n}x{k} r{rank} of {adapters} {kind}", exact=True)


def test_forward_without_ranks_and_scales():
    rng = np.random.default_rng(1)
    c = Case(rng, 50, 90, 110, 12, 4, "bf16", True)
    c.a, c.b = np.nan_to_num(c.a, nan=0.5), np.nan_to_num(c.b, nan=0.25)
    check_forward(c, "no ranks", ranks=False)
    check_forward(c, "no scales", scales=False)
    check_forward(c, "neither", ranks=False, scales=False)
    c.ranks[:] = [-4, 99, 12, 0]   # taken as 0, 12, 12, 0
    d = Case(rng, 50, 90, 110, 12, 4, "bf16", True)
    d.__dict__.update({n: getattr(c, n) for n in ("x", "c", "a", "b", "ids", "scales")}, ranks=np.array([0, 12, 12, 0], np.int32))
    say("ranks out of range")
    assert np.array_equal(run_forward(c), run_forward(d))


@pytest.mark.parametrize("kind", KINDS)
def test_rows_do_not_mix(kind):
    """A NaN or infinity in a row, or in an adapter, reaches that row and the rows of that
    adapter; a row without an adapter keeps every bit, -0 too. Infinities stay infinite."""
    rng = np.random.default_rng(6)
    c = Case(rng, 40, 70, 96, 8, 5, kind, True)
    c.ranks[:] = 8
    c.a, c.b = mxref.to_type(rng.normal(size=c.a.shape), KINDS[kind]), mxref.to_type(rng.normal(size=c.b.shape), KINDS[kind])
    c.ids = np.arange(40, dtype=np.int32) % 6 - 1          # every sixth has none
    clean = run_forward(c)
    c.x[3] = np.nan
    c.x[8, 5] = np.inf
    c.c[0], c.c[6] = -0.0, np.nan
    c.a[1, 2, 3] = np.nan
    c.b[2, 7, 1] = np.inf
    say(f"rows do not mix {kind}")
    y = run_forward(c)
    assert np.isnan(y[3]).all() and np.isnan(y[c.ids == 1]).all()
    assert (y[0] == 0).all() and np.signbit(y[0]).all() and np.isnan(y[6]).all()
    at2 = c.ids == 2
    assert not np.isfinite(y[at2, 7]).any()
    h = c.x.astype(np.float64) @ c.a[2, 1].astype(np.float64)
    for row in np.nonzero(at2 & np.isfinite(c.x).all(axis=1))[0]:
        assert y[row, 7] == np.inf * np.sign(h[row] * c.scales[2])
    assert not np.isfinite(y[8]).any()                     # an infinity times every column of A
    same = np.ones_like(y, bool)
    for row in range(40):
        if c.ids[row] == 1 or row in (0, 3, 6, 8):
            same[row] = False
        if c.ids[row] == 2:
            same[row, 7] = False
    assert np.array_equal(y[same], clean[same])


def run_backward(c, base="other", workspace=True, dx=True, weights=True, s=None):
    t = torch()
    s = s or c.set()
    x, ldx = padded(c.x, c.kind, c.pad, c.offset)
    dy, lddy = padded(c.dy, c.kind, c.pad + 1, c.offset)
    cd, ldc = padded(c.dc, c.kind, c.pad, c.offset, SENTINEL if base == "place" else np.nan)
    if base == "place":
        dxd, lddx = cd, ldc
    else:
        lddx = c.k + c.pad + 1
        dxd = t.full((c.rows * lddx + 8,), SENTINEL, device="cuda:0").to(dtype(c.kind))
    da = t.full((c.a.size + 8,), SENTINEL, device="cuda:0")
    db = t.full((c.b.size + 8,), SENTINEL, device="cuda:0")
    need = lib.gemm_lora_backward_workspace_bytes(c.rows, s)
    ws = t.full((need + 16,), 0xff, dtype=t.uint8, device="cuda:0") if workspace else None
    lib.gemm_lora_backward(c.rows, s, c.di, x, ldx, dy, lddy, None if base == "none" else cd, ldc, dxd if dx else None, lddx, da if weights else None,
                           db if weights else None, ws, need if workspace else 0, stream())
    out, da, db = host(dxd), host(da), host(db)
    assert (da[c.a.size:] == SENTINEL).all() and (db[c.b.size:] == SENTINEL).all()
    if workspace:
        assert (ws[need:] == 0xff).all()
    if dx:
        assert (out[c.rows * lddx:] == SENTINEL).all() or base == "place"
        out = out[:c.rows * lddx].reshape(c.rows, lddx)
        assert (out[:, c.k:] == SENTINEL).all()
        out = out[:, :c.k]
    else:
        assert base == "place" or (out == SENTINEL).all()
    if not weights:
        assert (da == SENTINEL).all() and (db == SENTINEL).all()
    return out, da[:c.a.size].reshape(c.a.shape), db[:c.b.size].reshape(c.b.shape)


def check_backward(c, what, base="other", workspace=True, exact=False, dx=True, weights=True):
    say(what)
    got = run_backward(c, base, workspace, dx, weights)
    want, mag = ref.lora_backward(c.x.astype(np.float64), c.dy.astype(np.float64), None if base == "none" else c.dc, c.a.astype(np.float64),
                                  c.b.astype(np.float64), c.ids, c.ranks, c.scales)
    # as forward; a sum over an adapter's rows takes up to 5 products of parts for each of them
    many = max([(c.ids == i).sum() for i in range(c.adapters)])
    terms = (c.n + 5 * c.rank + 40, c.n + 5 * many + 60, c.k + 5 * many + 60)
    for i, name in enumerate(("dx", "da", "db")):
        if not (dx if i == 0 else weights):
            continue
        kind = c.kind if i == 0 else "f32"
        if exact:
            assert np.array_equal(got[i], mxref.to_type(want[i], KINDS[kind])), (what, name)
            continue
        bound = mag[i] * terms[i] * 2.0 ** -23
        bound = bound + half_step(kind, np.abs(want[i]) + bound)
        assert (np.abs(got[i] - want[i]) <= bound).all(), (what, name, np.nanmax(np.abs(got[i] - want[i]) / np.maximum(bound, 1e-300)), np.isnan(got[i]).sum())


@pytest.mark.parametrize("rows,n,k,rank,adapters", SIZES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("mixed", [False, True])
def test_backward(rows, n, k, rank, adapters, kind, mixed):
    rng = np.random.default_rng(rows + n + k + rank)
    c = Case(rng, rows, n, k, rank, adapters, kind, mixed, pad=rows % 3, offset=n % 2)
    for base in ("other", "place", "none"):
        check_backward(c, f"lora backward {rows}x{n}x{k} r{rank} of {adapters} {kind} mixed {mixed} {base}", base, workspace=base != "none")


@pytest.mark.parametrize("rows,n,k,rank,adapters", SIZES)
@pytest.mark.parametrize("kind", KINDS)
def test_backward_whole_numbers(rows, n, k, rank, adapters, kind):
    rng = np.random.default_rng(rows * 7 + n)
    c = Case(rng, rows, min(n, 300), min(k, 300), rank, adapters, kind, True, whole=True, pad=1)
    check_backward(c, f"lora backward whole numbers {rows}x{n}x{k} r{rank} of {adapters} {kind}", exact=True)


@pytest.mark.parametrize("kind", KINDS)
def test_backward_of_some(kind):
    rng = np.random.default_rng(2)
    c = Case(rng, 90, 70, 130, 20, 4, kind, True)
    check_backward(c, f"only dX {kind}", weights=False)
    check_backward(c, f"only dX in place {kind}", base="place", weights=False)
    check_backward(c, f"only dA and dB {kind}", dx=False)
    c.ids[:] = -1
    c.a[:], c.b[:] = np.nan, np.nan
    check_backward(c, f"no row with an adapter {kind}")
    c = Case(rng, 90, 70, 130, 20, 1024, kind, True)
    check_backward(c, f"more adapters than rows {kind}")


def test_backward_without_rows():
    t = torch()
    c = Case(np.random.default_rng(2), 4, 30, 20, 5, 3, "f32", True)
    s = c.set()
    da, db = t.full((c.a.size,), SENTINEL, device="cuda:0"), t.full((c.b.size,), SENTINEL, device="cuda:0")
    lib.gemm_lora_backward(0, s, None, None, 20, None, 30, None, 20, None, 20, da, db, None, 0, stream())
    assert (da == 0).all() and (db == 0).all()


def test_backward_many_rows_of_one_adapter():
    """Several stretches of rows, whose sums are joined; whole numbers, so every bit counts."""
    rng = np.random.default_rng(3)
    c = Case(rng, 5000, 40, 600, 7, 2, "bf16", True, whole=True)
    check_backward(c, "5000 rows", exact=True)
    c = Case(rng, 5000, 600, 40, 70, 1, "f32", False)
    check_backward(c, "5000 rows FP32")


@pytest.mark.parametrize("kind", KINDS)
def test_backward_many_adapters(kind):
    """More tiles to transpose than workgroups; whole numbers, so every bit counts."""
    rng = np.random.default_rng(31)
    for mixed in (False, True):
        c = Case(rng, 900, 300, 260, 5, 1000, kind, mixed, whole=True)
        check_backward(c, f"900 rows on 1000 adapters {kind}", exact=True)
        check_backward(c, f"900 rows on 1000 adapters, no dX {kind}", exact=True, dx=False)


@pytest.mark.parametrize("kind", KINDS)
def test_same_bits_every_time(kind):
    rng = np.random.default_rng(9)
    c = Case(rng, 1500, 300, 260, 40, 5, kind, True)
    first = (run_forward(c),) + run_backward(c)
    for _ in range(3):
        again = (run_forward(c),) + run_backward(c)
        for p, q in zip(first, again):
            assert np.array_equal(p, q)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,rank", [(40, 8), (40, 100), (1500, 24)])
def test_gradients_do_not_mix(rows, rank, kind):
    """A NaN or infinity in a row reaches the gradients of that row and of its adapter, up to that
    adapter's own rank: behind it, and where no row has the adapter, they are zeros."""
    rng = np.random.default_rng(rows + rank)
    c = Case(rng, rows, 70, 96, rank, 6, kind, True)
    c.ranks[:] = [rank, 3, rank // 2, rank, 0, rank]
    c.a, c.b = mxref.to_type(rng.normal(size=c.a.shape), KINDS[kind]), mxref.to_type(rng.normal(size=c.b.shape), KINDS[kind])
    c.ids = np.arange(rows, dtype=np.int32) % 6 - 1        # every sixth has none; none has adapter 5
    clean = run_backward(c)
    c.x[0], c.dy[6] = np.nan, np.inf                       # of no adapter
    c.x[8], c.dy[14] = np.nan, np.inf                      # of adapter 1
    c.x[15], c.dy[9] = np.inf, np.nan                      # of adapter 2
    c.x[11], c.dy[5] = np.nan, np.inf                      # of adapter 4, rank 0
    say(f"gradients do not mix {rows} r{rank} {kind}")
    dx, da, db = run_backward(c)
    same = ~np.isin(np.arange(rows), [5, 6, 9, 14])
    assert np.array_equal(dx[same], clean[0][same])
    assert np.array_equal(dx[6], clean[0][6]) and np.array_equal(dx[5], clean[0][5])
    assert not np.isfinite(dx[[9, 14]]).any()
    for i in range(6):
        own = c.ranks[i]
        assert (da[i, own:] == 0).all() and (db[i, :, own:] == 0).all(), i
        if i in (1, 2):
            assert not np.isfinite(da[i, :own]).any() and not np.isfinite(db[i, :, :own]).any()
        else:
            assert np.array_equal(da[i], clean[1][i]) and np.array_equal(db[i], clean[2][i])
    assert (da[5] == 0).all() and (db[5] == 0).all()


def test_gradient_against_differences():
    """Differences of what gemm_lora itself gives: the sum of Y dY is linear in each input, so with whole
    numbers and steps of 1 the differences are exact."""
    rng = np.random.default_rng(4)
    c = Case(rng, 12, 10, 9, 3, 3, "f32", True, whole=True)
    dx, da, db = run_backward(c, base="none")

    def loss():
        return (run_forward(c, "none").astype(np.float64) * c.dy).sum()

    base = loss()
    for array, grad in ((c.x, dx), (c.a, da), (c.b, db)):
        for at in list(np.ndindex(*array.shape))[::7]:
            if np.isnan(array[at]):
                assert grad[at] == 0
                continue
            array[at] += 1
            assert loss() - base == grad[at], at
            array[at] -= 1


@pytest.mark.parametrize("kind,small,back", [("f16", -24, 14), ("bf16", -120, 110), ("f32", -120, 110)])
def test_small_values(kind, small, back):
    """Whole numbers times the smallest half (subnormal there), or near the smallest normal float: sums stay
    exact, and the scale brings them back."""
    rng = np.random.default_rng(10)
    c = Case(rng, 40, 70, 90, 10, 3, kind, True, whole=True)
    c.x, c.scales = c.x * np.float32(2.0 ** small), c.scales * np.float32(2.0 ** back)
    check_forward(c, f"small values {kind}", base="none", exact=True)
    c.dc[:] = 0
    c.dy, c.x = c.dy * np.float32(2.0 ** small), c.x * np.float32(2.0 ** -small)
    check_backward(c, f"small gradients {kind}", base="none", exact=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [63, 64, 65, 128, 129, 4096, 4159])
def test_row_counts_around_the_kernels_borders(rows, kind):
    """Windows of 64 rows, the layouts for few and many rows, units of two tiles with an odd one."""
    rng = np.random.default_rng(rows)
    for mixed in (False, True):
        c = Case(rng, rows, 130, 70, 18, 4, kind, mixed, whole=True, pad=2)
        check_forward(c, f"rows {rows} {kind} mixed {mixed}", base="place", exact=True)
        check_backward(c, f"rows {rows} {kind} mixed {mixed}", base="place", exact=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 4, 16, 17, 100, 127, 128, 129, 141, 144, 240, 255, 257, 400])
def test_columns_around_a_workgroups_last(n, kind):
    """Both products in one kernel where a workgroup's 128 columns end inside the matrix, inside a wave's 16 or
    before some of its waves begin: the waves share K and its barriers whatever they have to store."""
    rng = np.random.default_rng(n)
    for rows, rank in ((1, 7), (40, 16), (64, 32)):
        c = Case(rng, rows, n, 333, rank, 9, kind, True, whole=True, pad=n % 2)
        assert lib.gemm_lora_workspace_bytes(rows, c.set()) == 0   # (one kernel)
        for base in ("other", "place", "none"):
            check_forward(c, f"{n} columns, {rows} rows, rank {rank} {kind} {base}", base, exact=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,rank", [(4096, 48), (4159, 64), (4100, 33), (4159, 100), (4096, 128)])
def test_many_rows_of_large_ranks(rows, rank, kind):
    """Units of two tiles at every width above 32 ranks; whole numbers, so every bit counts."""
    rng = np.random.default_rng(rows + rank)
    for mixed in (False, True):
        c = Case(rng, rows, 150, 200, rank, 3, kind, mixed, whole=True, pad=1)
        check_forward(c, f"{rows} rows, rank {rank} {kind} mixed {mixed}", base="none" if mixed else "other", exact=True)
        check_backward(c, f"{rows} rows, rank {rank} {kind} mixed {mixed}", base="none" if mixed else "other", exact=True)


@pytest.mark.parametrize("rows", [2, 70])
def test_a_sum_near_the_largest_float_beside_an_infinite_row(rows):
    """A row whose H B^T stays below the largest float, though the first bfloat16 parts of H alone pass it, keeps its
    bits when another row of its adapter becomes infinite (which has the first parts looked at alone)."""
    c = Case(np.random.default_rng(1), rows, 17, 3, 5, 1, "bf16", True)
    c.ids[:], c.ranks[:], c.scales[:] = 0, 5, 1.0
    # H: twice -2^126 (1 + 2^-8 (1 - 2^-6)), whose first part is -2^126, and twice 1.5 2^127
    c.a[0] = [[-2.0 ** 126, -2.0 ** 118, 2.0 ** 112]] * 2 + [[1.5 * 2.0 ** 127, 0, 0]] * 2 + [[0, 0, 0]]
    c.b[:], c.x[0], c.x[1:] = 1.0, 1.0, 0.0
    c.c[:] = -2.0 ** 127
    say(f"a sum near the largest float, {rows} rows")
    clean = run_forward(c)
    c.x[1] = np.inf
    assert np.array_equal(run_forward(c)[0], clean[0])
    # 2^128 - 2^119 (1 - 2^-6) - 2^127, where a bfloat16's step is 2^119
    assert (clean[0] == 2.0 ** 127 - 2.0 ** 119).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [9, 300])
def test_backward_to_the_rows_without_x(rows, kind):
    """dX alone takes no X."""
    t = torch()
    c = Case(np.random.default_rng(rows), rows, 70, 90, 20, 4, kind, True)
    want = run_backward(c, base="none", weights=False)[0]
    s = c.set()
    dy, dx = dev(c.dy, kind), t.full((rows, c.k), SENTINEL, device="cuda:0").to(dtype(kind))
    say(f"dX without X {rows} {kind}")
    lib.gemm_lora_backward(rows, s, c.di, None, 0, dy, c.n, None, 0, dx, c.k, None, None, None, 0, stream())
    assert np.array_equal(host(dx), want)
