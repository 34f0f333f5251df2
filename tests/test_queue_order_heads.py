"""The pass-2 work queue of the post-training heads, checked on the host.

As in test_queue_order, with two differences: chunks are as wide as 64 MB of G
allow, and where dX has fewer tiles than there are SM pairs, each of its tiles
is several items, one per range of the chunk's vocabulary, with an fp32 sum of
its own.  An item of a range waits for what its tile waited for: its token tile's
G(c) row, and every range of dX(c-1) of that token tile.  G(c) waits for every range
of dX(c-1) of its token tile, and for dW(c-1) of its column.

The sizes are restated here and held to the library's workspace query."""
import itertools

import pytest

TILE, BK, VC = 256, 64, 2048
WIDE_G, WIDE_CHUNK, PAIRS = 64 << 20, 1 << 20, 74


def chunk_of(N, V):
    most = max(VC, min(WIDE_CHUNK, WIDE_G // (2 * N)) // TILE * TILE)
    chunks = -(-V // most)
    return max(VC, (-(-V // chunks) + TILE - 1) // TILE * TILE)


def ranges_of(N, H, V, chunk):
    tiles = -(-N // TILE) * -(-H // TILE)
    last = V % chunk or chunk
    most = min(-(-last // BK), max(1, min(V, chunk) // (16 * BK)))
    return max(1, min(PAIRS // tiles, most, 64))


def layout(N, H, V, wide=True):
    chunk = chunk_of(N, V) if wide else VC
    ks = ranges_of(N, H, V, chunk) if wide else 1
    TM, HN, C = -(-N // TILE), -(-H // TILE), -(-V // chunk)
    VT_last = -(-(V - (C - 1) * chunk) // TILE)
    VTf = chunk // TILE if C > 1 else VT_last
    rows = TM * VTf <= 3 * PAIRS
    return dict(N=N, H=H, V=V, chunk=chunk, KS=ks, TM=TM, HN=HN, HW=HN if rows else (HN + 1) // 2, C=C, VTf=VTf,
                VT_last=VT_last, cols_first=0 if rows else 1 << 20)


def vtiles(p, c):
    return p["VT_last"] if c == p["C"] - 1 else p["VTf"]


def section(p, c):
    n = p["TM"] * p["HN"] * p["KS"] + vtiles(p, c) * p["HW"]
    return n + (vtiles(p, c + 1) * p["TM"] if c + 1 < p["C"] else 0)


def grad(p, c, r):
    vt = vtiles(p, c)
    k = min(p["cols_first"], vt)
    if r < k * p["TM"]:
        return ("G", c, r % p["TM"], r // p["TM"])
    r -= k * p["TM"]
    return ("G", c, r // (vt - k), k + r % (vt - k))


def decode(p, i):
    """Item i as a tuple of (kind, chunk, row, column) tiles, dX with its range."""
    g0 = vtiles(p, 0) * p["TM"]
    if i < g0:
        return (grad(p, 0, i),)
    r, c = i - g0, 0
    if p["C"] >= 3:  # sections 0 .. C-3 have one size
        c = min(r // section(p, 0), p["C"] - 3)
        r -= c * section(p, 0)
    while c + 1 < p["C"] and r >= section(p, c):
        r -= section(p, c)
        c += 1
    nx, nw = p["TM"] * p["HN"] * p["KS"], vtiles(p, c) * p["HW"]
    if r < nx:
        a, b = divmod(r, p["HN"] * p["KS"])
        return (("X", c, a, b // p["KS"], b % p["KS"]),)
    if r < nx + nw:
        a, b = divmod(r - nx, p["HW"])
        if p["HW"] == p["HN"]:
            return (("W", c, a, b),)
        return tuple(("W", c, a, h) for h in (2 * b, 2 * b + 1) if h < p["HN"])
    return (grad(p, c + 1, r - nx - nw),)


def every_tile(p):
    for c in range(p["C"]):
        yield from (("G", c, t, v) for t, v in itertools.product(range(p["TM"]), range(vtiles(p, c))))
        yield from (("X", c, t, h, k) for t, h, k in itertools.product(range(p["TM"]), range(p["HN"]), range(p["KS"])))
        yield from (("W", c, v, h) for v, h in itertools.product(range(vtiles(p, c)), range(p["HN"])))


SHAPES = [
    (1, 8, 1), (1, 64, 300), (5, 16, 33), (256, 256, 4096), (300, 264, 5003), (515, 136, 2049), (700, 64, 9000),
    (700, 64, 60000), (3, 1024, 30000), (260, 520, 20011), (513, 136, 70001), (16, 4096, 128256), (512, 1024, 50000),
    (1024, 2304, 256000), (2048, 2304, 256000), (2048, 4096, 128256), (8192, 4096, 128256), (16384, 64, 2049),
    (20000, 72, 4097), (33000, 8, 2305), (256, 8, 1 << 21), (7000, 136, 12345),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("wide", [True, False])
def test_queue_drains(shape, wide):
    p = layout(*shape, wide)
    T = vtiles(p, 0) * p["TM"] + sum(section(p, c) for c in range(p["C"]))
    pos = {}
    for i in range(T):
        for t in decode(p, i):
            assert t not in pos
            pos[t] = i
    assert set(pos) == set(every_tile(p))
    # the last item of each group that something waits for
    g_row, x_row, g_col, w_col = {}, {}, {}, {}
    for t, i in pos.items():
        for table, key in {"G": ((g_row, t[1:3]), (g_col, (t[1], t[3]))), "X": ((x_row, t[1:3]),),
                           "W": ((w_col, t[1:3]),)}[t[0]]:
            table[key] = max(table.get(key, -1), i)
    for t, i in pos.items():
        kind, c, a, b = t[:4]
        if kind == "X":
            assert g_row[c, a] < i and (c == 0 or x_row[c - 1, a] < i)
        elif kind == "W":
            assert g_col[c, a] < i
        elif c:
            assert x_row[c - 1, a] < i and w_col[c - 1, b] < i


@pytest.mark.parametrize("shape", SHAPES)
def test_ranges_of_dx_cover_every_chunk(shape):
    """Each chunk's k-blocks once, and none of the ranges empty: an item without a
    k-block would have no accumulator to read."""
    p = layout(*shape)
    for c in {0, p["C"] - 1}:
        width = min(p["chunk"], p["V"] - c * p["chunk"])
        kblocks = -(-width // BK)
        ends = [kblocks * k // p["KS"] for k in range(p["KS"] + 1)]
        assert ends[0] == 0 and ends[-1] == kblocks and all(a < b for a, b in zip(ends, ends[1:]))


@pytest.mark.parametrize("shape", SHAPES)
def test_sizes_are_the_library_s(shape):
    import __graft_entry__
    __graft_entry__.build()
    import lm_head_linear_03_b200 as F
    N, H, V = shape
    p = layout(N, H, V)

    def up(n):
        return (n + 255) // 256 * 256

    def areas(chunk, ks):
        return (up((2 * p["TM"] + 2 * (chunk // TILE)) * 4) + up(N * chunk * 2)
                + (up(N * H * 4 * ks) if ks > 1 else 0))

    assert F.policy_workspace_size(N, H, V) - F.workspace_size(N, H) == areas(p["chunk"], p["KS"]) - areas(VC, 1)
