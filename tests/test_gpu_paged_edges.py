"""The paged memory cache's calls at the edges of what they take: values that are not finite or of extreme size, calls
that are refused half way, token ranges that are none.  Against float64 numpy (paged_reference.py)."""
import numpy as np
import pytest
import torch

from mamba_ssd_state_b200 import dart
from tests import paged_reference as ref
from tests.parity import rel_err
from tests.test_gpu_paged import SHAPES, TOL, Pool, attention_inputs, cast, cumulative, extend_inputs, ints, memories_of, states

pytestmark = pytest.mark.gpu
FOUR_BIT = [v for v in SHAPES if v[3] == "mxfp4"]


# ------------------------------------------- 4-bit blocks that are no numbers
@pytest.mark.parametrize("N, P, dtype, cache, H, G", FOUR_BIT)
@pytest.mark.parametrize("lens", [[1], [2], [4], [5], [8], [3, 7]])
@pytest.mark.parametrize("row", [0, 1, 7, 8, 9, 34, 63])
def test_a_scale_of_255_is_nan_for_every_token_that_sees_it(N, P, dtype, cache, H, G, lens, row):
    """Blocks from elsewhere may have codes that are not zero beside the scale byte 255; whichever column holds the
    block and whichever token sees it, even or odd, its readout is NaN."""
    rng = np.random.default_rng(row + sum(lens))
    memories = memories_of(rng, [6] * len(lens), H, N, P, cache, scale=0.5)
    pool = Pool(memories, H, N, P, 4, cache, rng)
    for b in range(len(lens)):
        pool.scales[pool.table_np[b, 0], :, 3, row, (row + b) % (N // 32)] = 255
    T = sum(lens)
    args, args64 = attention_inputs(rng, T, H, G, N, P, dtype)
    for sees in (lambda t: t % 2 == 0, lambda t: t % 2 == 1, lambda t: True):
        see = np.array([bool(sees(t)) for t in range(T)])
        counts = np.where(see, 6, 3).tolist()
        out = dart.dart_sma_paged(*args, cumulative(lens), pool.pages, pool.table, ints(*counts), 1.0, scales=pool.scales)
        dart.dart_sync_status()
        want = ref.sma(*args64, lens, memories, [3] * T)
        assert torch.isnan(out[torch.from_numpy(see).cuda()]).all()
        assert rel_err(out[torch.from_numpy(~see).cuda()], want[~see]) <= TOL if (~see).any() else True


# --------------------------------------------------- the range of the scales
@pytest.mark.parametrize("N, P, dtype, cache, H, G", FOUR_BIT)
@pytest.mark.parametrize("lens", [[1], [3], [8], [2, 6]])
@pytest.mark.parametrize("low, high, q, c", [(0, 0, 125, 90), (0, 3, 124, 100), (222, 228, -101, -80), (240, 250, -122, -112),
                                             (250, 252, -124, -115)])
def test_attention_over_the_whole_range_of_scale_bytes(N, P, dtype, cache, H, G, lens, low, high, q, c):
    """Scale bytes at both ends of what float32 holds, and tokens that bring scores and values back to ordinary size."""
    rng = np.random.default_rng(low + sum(lens))
    pool = Pool(memories_of(rng, [7] * len(lens), H, N, P, cache, scale=0.5), H, N, P, 3, cache, rng)
    held = []
    for b in range(len(lens)):
        for m in range(7):
            scales = rng.integers(low, high + 1, (H, P, N // 32)).astype(np.uint8)
            pool.scales[pool.table_np[b, m // 3], :, m % 3] = torch.from_numpy(scales).cuda()
        held.append(np.stack([pool.memory(b, m) for m in range(7)]))
    T = sum(lens)
    Q, Q64 = cast(rng.standard_normal((T, H, N)) * 2.0 ** q, dtype)
    E, E64 = cast(rng.standard_normal((T, H, P)) / np.sqrt(P), dtype)
    C, C64 = cast(rng.standard_normal((T, G, N)) * 2.0 ** c, dtype)
    counts = [7 - (t % 3) for t in range(T)]
    want = ref.sma(Q64, E64, C64, lens, held, counts)
    out = dart.dart_sma_paged(Q, E, C, cumulative(lens), pool.pages, pool.table, ints(*counts), 1.0, scales=pool.scales)
    dart.dart_sync_status()
    # TOL counts for scores of up to 12, whose error goes with their size
    ends = np.cumsum([0] + lens)
    size = max(np.abs(np.einsum("thn,mhnp,thp->thm", Q64[a:e], m, E64[a:e])).max() / np.sqrt(N)
               for m, a, e in zip(held, ends[:-1], ends[1:]))
    assert rel_err(out, want) <= TOL * max(1.0, size / 12)


@pytest.mark.parametrize("N, P, dtype, cache, H, G", FOUR_BIT)
def test_many_sequences_over_scales_of_all_kinds(N, P, dtype, cache, H, G):
    """Items that one worker does whole, with and without y_ssd; the last memory's blocks are NaN."""
    rng = np.random.default_rng(31)
    B = 1200
    lens = [int(v) for v in rng.integers(0, 4, B)]
    T = sum(lens)
    pool = Pool(memories_of(rng, [4], H, N, P, cache, scale=0.5), H, N, P, 2, cache, rng)
    for m in range(3):
        scales = rng.integers(220, 228, (H, P, N // 32)).astype(np.uint8)
        pool.scales[pool.table_np[0, m // 2], :, m % 2] = torch.from_numpy(scales).cuda()
    pool.scales[pool.table_np[0, 1], :, 1, ::2] = 255
    held = np.stack([pool.memory(0, m) for m in range(3)])
    pool.table = pool.table.expand(B, 2).contiguous()             # all read the same pages
    Q, Q64 = cast(rng.standard_normal((T, H, N)) * 2.0 ** -100, dtype)
    E, E64 = cast(rng.standard_normal((T, H, P)) / np.sqrt(P), dtype)
    C, C64 = cast(rng.standard_normal((T, G, N)) * 2.0 ** -104, dtype)
    y, y64 = cast(rng.standard_normal((T, H, P)), "f32")
    counts = rng.integers(0, 5, T)
    o = ref.sma(Q64, E64, C64, lens, [held] * B, np.minimum(counts, 3).tolist())
    out = dart.dart_sma_paged(Q, E, C, cumulative(lens), pool.pages, pool.table, ints(*counts.tolist()), 0.5, y, scales=pool.scales)
    bare = dart.dart_sma_paged(Q, E, C, cumulative(lens), pool.pages, pool.table, ints(*counts.tolist()), 0.5, scales=pool.scales)
    dart.dart_sync_status()
    fine = torch.from_numpy(counts < 4).cuda()
    assert torch.isnan(out[~fine]).all() and torch.isnan(bare[~fine]).all()
    assert rel_err(out[fine], (y64 + 0.5 * o)[counts < 4]) <= TOL and rel_err(bare[fine], o[counts < 4]) <= TOL


# ------------------------------------------------- tokens that are no numbers
@pytest.mark.parametrize("N, P, dtype", [(128, 64, "bf16"), (64, 64, "bf16"), (128, 64, "f32"), (64, 64, "f32"), (16, 16, "bf16")])
@pytest.mark.parametrize("lens, S", [([70], 64), ([70], 256), ([30, 45], 32), ([12, 40, 12], 48), ([9, 14], 256)])
@pytest.mark.parametrize("what", ["x", "dt", "B", "C", "x last"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_token_that_is_not_finite_leaves_earlier_ones_alone(N, P, dtype, lens, S, what, value):
    """The recurrence is causal for every value, in runs of any length: what a token holds reaches its own output and
    later ones, no earlier one, no other head and, of x, no other column."""
    rng = np.random.default_rng(sum(lens) + N)
    H, B = 3, len(lens)
    pool = Pool([[]] * B, H, N, P, 2, "bf16" if dtype == "bf16" else "f32", rng, room=1 + max(lens) // S)
    args, args64 = extend_inputs(rng, lens, H, 1, N, P, dtype)
    s, c, s64, c64 = states(rng, B, H, N, P)
    n, pos = [0] * B, [S // 2] * B
    yr, sr, cr, *_ = ref.extend(*args64, lens, s64, c64, n, pos, S)
    x, dt, A, Bm, Cm = args
    b, h, p = B - 1, 1, P - 3
    at = lens[b] - 1 if what == "x last" else lens[b] // 2 | 1          # odd: the second of two tokens that share a lane
    t = sum(lens[:b]) + at
    end = sum(lens)
    touched = np.zeros((end, H, P), bool)
    if what in ("x", "x last"):
        x[t, h, p] = value
        touched[t:, h, p] = True
    elif what == "dt":
        dt[t, h] = value
        touched[t:, h] = True
    elif what == "B":
        Bm[t, 0, N // 2] = value
        touched[t:] = True
    else:
        Cm[t, 0, N // 2] = value
        touched[t] = True
    got = dart.dart_ssd_extend(x, dt, A, Bm, Cm, cumulative(lens), s, c, pool.pages, pool.table, ints(*n), ints(*pos), S)
    dart.dart_sync_status()
    y = got["y"].cpu().double().numpy()
    assert rel_err(np.where(touched, 0.0, y), np.where(touched, 0.0, yr)) <= TOL
    assert not np.isfinite(y[touched]).any()
    for key, want in (("state", sr), ("dH_cur", cr)):
        v = got[key].cpu().double().numpy()
        kept = np.ones_like(v, bool)
        if what in ("x", "x last"):
            kept[b, h, :, p] = False
        elif what == "dt":
            kept[b, h] = False
        elif what == "B":
            kept[b, :, N // 2] = False
        assert rel_err(np.where(kept, v, 0.0), np.where(kept, want, 0.0)) <= TOL


@pytest.mark.parametrize("N, P, dtype", [(128, 64, "bf16"), (64, 64, "bf16"), (128, 64, "f32"), (16, 16, "bf16")])
@pytest.mark.parametrize("lens", [[70], [9]])
def test_a_token_that_forgets_everything_leaves_earlier_ones_alone(N, P, dtype, lens):
    """dt A of -1e30: what comes before it keeps its decays."""
    rng = np.random.default_rng(3)
    H, S, at = 2, 256, lens[0] // 2 | 1
    pool = Pool([[]], H, N, P, 2, "bf16" if dtype == "bf16" else "f32", rng, room=1)
    (x, dt, A, Bm, Cm), args64 = extend_inputs(rng, lens, H, 1, N, P, dtype)
    s, c, s64, c64 = states(rng, 1, H, N, P)
    yr = ref.extend(*args64, lens, s64, c64, [0], [0], S)[0]
    dt[at] = 1e30
    got = dart.dart_ssd_extend(x, dt, A, Bm, Cm, cumulative(lens), s, c, pool.pages, pool.table, ints(0), ints(0), S)
    dart.dart_sync_status()
    assert rel_err(got["y"][:at], yr[:at]) <= TOL


# ------------------------------------------------- calls that are refused
def test_a_layer_call_that_is_refused_changes_nothing():
    """layer_extend is two operators; whatever the second one refuses is refused before the first one runs."""
    rng = np.random.default_rng(5)
    H, N, P, S, lens = 2, 64, 64, 4, [3, 2]
    pool = Pool([[], []], H, N, P, 2, "bf16", rng, room=2)
    (x, dt, A, Bm, Cm), _ = extend_inputs(rng, lens, H, 1, N, P, "bf16")
    (Q, E, _), _ = attention_inputs(rng, 5, H, 1, N, P, "bf16")
    s, c, _, _ = states(rng, 2, H, N, P)
    n, pos = ints(0, 1), ints(2, 3)
    before = [v.clone() for v in (s, c, pool.pages.view(torch.int16), n, pos)]
    odd = lambda v: torch.cat((v.new_zeros(1), v.flatten()))[1:].reshape(v.shape)      # contiguous, at an address of its own
    ok = dict(x=x, dt=dt, A=A, Bm=Bm, Cm=Cm, Q=Q, E=E, g=0.5, cu_tokens=cumulative(lens), state=s, dH_cur=c, pages=pool.pages,
              table=pool.table, nchunks=n, pos=pos, chunk=S)
    T = 16400                                          # more than an attention call takes
    (x2, dt2, _, B2, C2), _ = extend_inputs(rng, [T], H, 1, N, P, "bf16")
    many = dict(x=x2, dt=dt2, Bm=B2, Cm=C2, Q=torch.zeros((T, H, N), dtype=torch.bfloat16, device="cuda"),
                E=torch.zeros((T, H, P), dtype=torch.bfloat16, device="cuda"))
    for kw in (dict(Q=Q.float()), dict(E=E.float()), dict(Q=Q[:4]), dict(E=E[:4]), dict(Q=Q[..., :32].contiguous()), dict(E=E[:, :1]),
               dict(E=E[..., :32]), dict(Q=odd(Q)), dict(E=odd(E)), dict(g="half"), dict(Q=Q[:, :1]), dict(Q=Q[0]), dict(E=E[0, 0]), many):
        with pytest.raises((TypeError, ValueError, dart.DartError)):
            dart.layer_extend(**{**ok, **kw})
        dart.dart_sync_status()
        for was, v in zip(before, (s, c, pool.pages.view(torch.int16), n, pos)):
            assert torch.equal(was, v)
    dart.layer_extend(**ok)
    dart.dart_sync_status()
    assert not torch.equal(before[0], s)


@pytest.mark.parametrize("cache", ["bf16", "mxfp4"])
def test_neighbours_in_one_buffer_are_apart(cache):
    """Every tensor of both calls is a slice of one buffer, one right behind the other."""
    rng = np.random.default_rng(6)
    H, N, P, S, R, lens, mems = 2, 128, 64, 4, 2, [3, 2], [1, 2]
    memories = memories_of(rng, mems, H, N, P, cache, scale=0.5)
    pool = Pool(memories, H, N, P, R, cache, rng, room=2)
    (x, dt, A, Bm, Cm), args64 = extend_inputs(rng, lens, H, 1, N, P, "bf16")
    (Q, E, _), (Q64, E64, _) = attention_inputs(rng, 5, H, 1, N, P, "bf16")
    s, c, s64, c64 = states(rng, 2, H, N, P)
    empty = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="cuda")
    i32 = torch.int32
    parts = dict(x=x, y=empty(5, H, P), dt=dt, mem_count=empty(5, dtype=i32), Bm=Bm, nchunks_out=empty(2, dtype=i32), Cm=Cm,
                 pos_out=empty(2, dtype=i32), cu_tokens=cumulative(lens), state=s, state_out=empty(*s.shape), dH_cur=c,
                 dH_cur_out=empty(*c.shape), pages=pool.pages, table=pool.table, nchunks=ints(*mems), pos=ints(1, 3), A=A, Q=Q,
                 out=empty(5, H, P), E=E, workspace=empty(dart.load().dart_sma_paged_workspace_bytes(dart._pack_dims(2, 5, H, P, N, 1, 1)) // 4))
    if pool.scales is not None:
        parts["scales"] = pool.scales
    size = lambda v: -(-v.numel() * v.element_size() // 16) * 16
    whole = torch.zeros(sum(size(v) for v in parts.values()), dtype=torch.uint8, device="cuda")
    at = 0
    for k, v in parts.items():
        there = whole[at:at + v.numel() * v.element_size()].view(v.dtype).view(v.shape)
        there.copy_(v)
        at += size(v)
        parts[k] = there
    pool.pages, pool.scales = parts["pages"], parts.get("scales")
    ext = ("x", "dt", "A", "Bm", "Cm", "cu_tokens", "state", "dH_cur", "pages", "table", "nchunks", "pos")
    outs = ("state_out", "dH_cur_out", "nchunks_out", "pos_out", "y", "mem_count")
    got = dart.dart_ssd_extend(*(parts[k] for k in ext), S, scales=pool.scales, **{k: parts[k] for k in outs})
    dart.dart_sma_paged(parts["Q"], parts["E"], parts["Cm"], parts["cu_tokens"], pool.pages, parts["table"], parts["mem_count"], 0.5,
                        parts["y"], scales=pool.scales, out=parts["out"], workspace=parts["workspace"])
    dart.dart_sync_status()
    yr, sr, cr, nr, pr, counts, _ = ref.extend(*args64, lens, s64, c64, mems, [1, 3], S)
    held = [np.stack([pool.memory(b, m) for m in range(nr[b])]) for b in range(2)]
    o = ref.sma(Q64, E64, args64[4], lens, held, counts)
    assert rel_err(parts["out"], yr + 0.5 * o) <= TOL
    assert rel_err(parts["state_out"], sr) <= TOL and rel_err(parts["dH_cur_out"], cr) <= TOL
    assert got["nchunks"].tolist() == nr and got["pos"].tolist() == pr and got["mem_count"].tolist() == counts
    assert torch.equal(parts["state"], s) and torch.equal(parts["dH_cur"], c) and torch.equal(parts["x"], x)


# ------------------------------------------------- token ranges that are none
def owned(cu, T):
    """The sequences that own their rows, by the rule of the header."""
    good = []
    for b in range(len(cu) - 1):
        before = [v for v in cu[:b] if 0 <= v <= T]
        good.append(0 <= cu[b] <= cu[b + 1] <= T and all(v <= cu[b] for v in before))
    return good


FALLING = [n if n != 650 else 600 for n in range(701)]      # sequence 650 would begin among the rows of 600 to 648
RANGES = [([0, 5, 3, 8], 9), ([-2, 3, 6], 8), ([0, 4, 99], 8), ([0, 99, 3, 8], 9), ([6, 8, 0, 4], 9), ([0, 40, 30, 70, 20, 90], 95),
          ([0, 300, 200, 500], 520), ([2, 2, 1, 1, 5], 6), (FALLING, 700)]


def test_the_ranges_of_these_tests():
    assert owned([0, 5, 3, 8], 9) == [True, False, False] and owned([0, 99, 3, 8], 9) == [False, False, True]
    assert owned([-2, 3, 6], 8) == [False, True] and owned([0, 4, 99], 8) == [True, False]
    assert [b for b, v in enumerate(owned(FALLING, 700)) if not v] == [649, 650]


@pytest.mark.parametrize("N, P, dtype, cache, H, G", SHAPES)
@pytest.mark.parametrize("cu, T", RANGES)
def test_attention_leaves_sequences_that_own_no_rows(N, P, dtype, cache, H, G, cu, T):
    rng = np.random.default_rng(T)
    B, good = len(cu) - 1, owned(cu, T)
    one = memories_of(rng, [4], H, N, P, cache, scale=0.5)[0]
    pool = Pool([one], H, N, P, 2, cache, rng)
    pool.table = pool.table.expand(B, 2).contiguous()
    args, args64 = attention_inputs(rng, T, H, G, N, P, dtype)
    counts = rng.integers(0, 5, T)
    rows = np.concatenate([np.arange(cu[b], cu[b + 1]) for b in range(B) if good[b]] + [np.arange(0)])
    y, y64 = cast(rng.standard_normal((T, H, P)), "f32")
    want = np.full((T, H, P), 5.0)
    want[rows] = y64[rows] + 0.5 * ref.sma(*[v[rows] for v in args64], [1] * len(rows), [one] * len(rows), counts[rows].tolist())
    out = torch.full_like(y, 5.0)
    out[rows] = y[rows]                                  # in place over y_ssd: nothing may be added twice
    dart.dart_sma_paged(*args, ints(*cu), pool.pages, pool.table, ints(*counts.tolist()), 0.5, out, scales=pool.scales, out=out)
    with pytest.raises(dart.DartError):
        dart.dart_sync_status()
    assert rel_err(out, want) <= TOL


MANY = [24 * n if n != 1050 else 24 * 1030 for n in range(1101)]


@pytest.mark.parametrize("N, P, dtype, H, cu, T", [(N, P, dtype, 2, cu, T) for N, P, dtype in [(128, 64, "bf16"), (64, 64, "f32"), (16, 16, "f32")]
                                                   for cu, T in RANGES] + [(64, 64, "bf16", 1, MANY, MANY[-1]), (16, 16, "f32", 1, MANY, MANY[-1])])
def test_recurrence_leaves_sequences_that_own_no_rows(N, P, dtype, H, cu, T):
    rng = np.random.default_rng(T)
    S, B, good = 64, len(cu) - 1, owned(cu, T)
    pool = Pool([[]] * B, H, N, P, 2, dtype, rng, room=5)
    args, args64 = extend_inputs(rng, [T], H, 1, N, P, dtype)
    s, c, s64, c64 = states(rng, B, H, N, P)
    y = torch.full((T, H, P), 9.0, device="cuda")
    seen = torch.full((T,), 99, dtype=torch.int32, device="cuda")
    got = dart.dart_ssd_extend(*args, ints(*cu), s.clone(), c.clone(), pool.pages, pool.table, ints(*[0] * B), ints(*[60] * B), S, y=y,
                               mem_count=seen)
    with pytest.raises(dart.DartError):
        dart.dart_sync_status()
    lens = [cu[b + 1] - cu[b] if good[b] else 0 for b in range(B)]
    rows = np.concatenate([np.arange(cu[b], cu[b + 1]) for b in range(B) if good[b]] + [np.arange(0)])
    yr, sr, cr, nr, pr, counts, _ = ref.extend(*[v[rows] if v.ndim > 1 else v for v in args64], lens, s64, c64, [0] * B, [60] * B, S)
    want, marks = np.full((T, H, P), 9.0), np.full(T, 99)
    want[rows], marks[rows] = yr, counts
    assert rel_err(y, want) <= TOL
    # rows of a sequence that has them in order and to itself, but begins before an earlier entry, stay as they are too
    assert (seen.cpu().numpy() == marks).all()
    assert rel_err(got["state"], sr) <= TOL and rel_err(got["dH_cur"], cr) <= TOL
    assert got["nchunks"].tolist() == nr and got["pos"].tolist() == pr


@pytest.mark.parametrize("N, P, dtype, cache, H, G", SHAPES)
@pytest.mark.parametrize("lens", [[1, 1], [4], [8], [3, 40], [200]])
@pytest.mark.parametrize("what", ["Q", "E", "C"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_row_that_is_not_finite_leaves_other_rows_alone(N, P, dtype, cache, H, G, lens, what, value):
    """One value of one token, in one head of Q or E or in one group of C: every other row of the tile is as it was."""
    rng = np.random.default_rng(sum(lens) + N)
    memories = memories_of(rng, [9] * len(lens), H, N, P, cache, scale=0.5)
    pool = Pool(memories, H, N, P, 4, cache, rng)
    T = sum(lens)
    (Q, E, C), args64 = attention_inputs(rng, T, H, G, N, P, dtype)
    counts = [9 - (t % 3) for t in range(T)]
    want = ref.sma(*args64, lens, memories, counts)
    t, touched = T // 2, np.zeros((T, H), bool)
    {"Q": Q, "E": E, "C": C}[what][t, -1, 5] = value
    touched[t, H - 1 if what != "C" else slice(H - H // G, H)] = True
    out = dart.dart_sma_paged(Q, E, C, cumulative(lens), pool.pages, pool.table, ints(*counts), 1.0, scales=pool.scales)
    dart.dart_sync_status()
    assert rel_err(out[torch.from_numpy(~touched).cuda()], want[~touched]) <= TOL
