"""The paged memory cache on the GPU against float64 numpy (paged_reference.py): writing and reading pages, the
recurrence over runs of tokens, the attention over pages, and all of them together as a server uses them."""
import numpy as np
import pytest
import torch

from mamba_ssd_state_b200 import dart, synth
from tests import paged_reference as ref
from tests.parity import rel_err

pytestmark = pytest.mark.gpu

# Products of bfloat16 or float32 inputs are summed in float32 (unit u = 2^-24), 200 or so terms to a sum.  The error
# of such a sum walks to about sqrt(200) u = 8e-7 of the root of its terms' squares; a score of size up to 12 is then
# off by 1e-5, the weight exp(score) by that much of itself, and the readout by no more.  The recurrence multiplies up
# to 80 factors exp(dt A), each good to 2 u: 80 * 2 * 6e-8 = 1e-5.  Both leave a factor of 2 to the largest value:
TOL = 2e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().cpu().double().numpy()


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Pool:
    """Pages scattered over a pool that is NaN wherever no memory was written."""

    def __init__(self, memories, H, N, P, R, cache, rng, spare=2, room=0):
        # memories: for every sequence [M, H, N, P] float64, already representable in the cache's format
        self.R, self.cache, self.N = R, cache, N
        need = [-(-(len(m) + room) // R) for m in memories]
        npages = sum(need) + spare
        order = rng.permutation(npages)
        width = max(1, max(need))
        self.table_np = np.full((len(memories), width), -1)
        if cache == "mxfp4":
            self.pages = torch.full((npages, H, R, P, N // 2), 0x77, dtype=torch.uint8, device="cuda")
            self.scales = torch.full((npages, H, R, P, N // 32), 255, dtype=torch.uint8, device="cuda")
        else:
            self.pages = torch.full((npages, H, R, N, P), float("nan"), dtype=DTYPES[cache], device="cuda")
            self.scales = None
        at = 0
        for b, mem in enumerate(memories):
            self.table_np[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            for m in range(len(mem)):
                page, slot = self.table_np[b, m // R], m % R
                if cache == "mxfp4":
                    codes, scales = ref.quantize(mem[m])
                    self.pages[page, :, slot] = torch.from_numpy(codes).cuda()
                    self.scales[page, :, slot] = torch.from_numpy(scales).cuda()
                else:
                    self.pages[page, :, slot] = torch.from_numpy(mem[m]).to(DTYPES[cache]).cuda()
        self.table = torch.from_numpy(self.table_np.astype(np.int32)).cuda()

    def memory(self, b, m):
        page, slot = self.table_np[b, m // self.R], m % self.R
        if self.cache == "mxfp4":
            return ref.dequantize(self.pages[page, :, slot].cpu().numpy(), self.scales[page, :, slot].cpu().numpy())
        return f64(self.pages[page, :, slot])


def memories_of(rng, counts, H, N, P, cache, scale=None):
    out = []
    for c in counts:
        m = rng.standard_normal((c, H, N, P)) * (N ** -0.5 if scale is None else scale)
        if cache == "mxfp4":
            m = ref.dequantize(*ref.quantize(m)) if c else m
        else:
            m = torch.from_numpy(m).to(DTYPES[cache]).double().numpy()
        out.append(m)
    return out


def cast(a, dtype):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DTYPES[dtype])
    return t.cuda(), t.double().numpy()


def cumulative(lens):
    return ints(*np.concatenate([[0], np.cumsum(lens)]).tolist())


# ------------------------------------------------------------ write and read
@pytest.mark.parametrize("N, P", [(128, 64), (64, 64), (16, 16)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R", [1, 3, 16])
def test_pages_hold_what_was_written(N, P, dtype, R):
    rng = np.random.default_rng(R)
    H, C, first, count = 3, 5, [0, 2, 1, 4], [5, 3, 0, 1]
    pool = Pool([[]] * 4, H, N, P, R, dtype, rng, room=8)
    before = pool.pages.clone()
    dH, want = cast(rng.standard_normal((4, H, C, N, P)), dtype)
    dart.dart_cache_write_paged(dH, ints(*first), ints(*count), pool.pages, pool.table)
    out = torch.full_like(dH, 7.0)
    dart.dart_cache_read_paged(pool.pages, pool.table, ints(*first), ints(*count), out=out)
    dart.dart_sync_status()
    for b in range(4):
        for i in range(count[b]):
            m = first[b] + i
            assert np.array_equal(pool.memory(b, m), want[b, :, i])
            before[pool.table_np[b, m // R], :, m % R] = dH[b, :, i]
            assert torch.equal(out[b, :, i], dH[b, :, i])
        assert (out[b, :, count[b]:] == 7.0).all()
    assert torch.equal(before.view(torch.uint8), pool.pages.view(torch.uint8))   # nothing else was touched


def hard_values(rng, shape, N):
    """Blocks with ties, zeros of both signs, one odd value out, tiny, huge, infinite and NaN values."""
    V = rng.standard_normal(shape)
    V[0, 0, 0, :8, 0] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    V[0, 0, 0, 8:32, 0] = 0.0
    V[0, 0, 0, :32, 1] = 0.0
    V[0, 0, 0, :32, 2] = -0.0
    V[0, 0, 1, :, 3] *= 2.0 ** -130
    V[0, 0, 1, :, 4] *= 2.0 ** 120
    V[0, 0, 1, 5, 4] = -(2.0 ** 127) * 1.5
    V[0, 0, 1, 7, 5], V[0, 0, 1, N - 1, 6], V[0, 0, 1, 0, 7] = np.nan, np.inf, -np.inf
    V[0, 0, 1, :, 8] = 3.0
    V[0, 0, 1, 4, 8] = 6.0
    V[0, 0, 1, :, 9] = np.where(np.arange(N) % 2, 6.0000005, -2.4999998)
    return V


@pytest.mark.parametrize("N", [128, 64])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R", [1, 5])
def test_four_bit_pages_are_the_nearest_codes(N, dtype, R):
    """Bit for bit: scales are powers of two, so that dividing by them rounds nothing."""
    rng = np.random.default_rng(10 + R)
    H, C, P, count = 2, 3, 64, [3, 2]
    pool = Pool([[]] * 2, H, N, P, R, "mxfp4", rng, room=4)
    dH, want = cast(hard_values(rng, (2, H, C, N, P), N), dtype)
    dart.dart_cache_write_paged(dH, ints(1, 0), ints(*count), pool.pages, pool.table, scales=pool.scales)
    out = torch.zeros_like(dH)
    dart.dart_cache_read_paged(pool.pages, pool.table, ints(1, 0), ints(*count), out=out, scales=pool.scales)
    dart.dart_sync_status()
    for b in range(2):
        for i in range(count[b]):
            m = i + (1 - b)
            codes, scales = ref.quantize(want[b, :, i])
            page, slot = pool.table_np[b, m // R], m % R
            assert np.array_equal(pool.scales[page, :, slot].cpu().numpy(), scales)
            assert np.array_equal(pool.pages[page, :, slot].cpu().numpy(), codes)
            read = torch.from_numpy(ref.dequantize(codes, scales)).to(DTYPES[dtype])
            assert torch.equal(torch.nan_to_num(out[b, :, i].cpu(), 123.0), torch.nan_to_num(read, 123.0))


def test_four_bit_scale_bytes_from_elsewhere():
    """All 256 scale bytes read as the format says, those that the library does not write too."""
    scales = torch.arange(256, dtype=torch.uint8, device="cuda").reshape(1, 1, 1, 64, 4).contiguous()
    pages = torch.randint(0, 256, (1, 1, 1, 64, 64), dtype=torch.uint8, device="cuda")
    out = torch.empty((1, 1, 1, 128, 64), device="cuda")
    dart.dart_cache_read_paged(pages, ints(0).reshape(1, 1), ints(0), ints(1), out=out, scales=scales)
    dart.dart_sync_status()
    want = ref.dequantize(pages.cpu().numpy(), scales.cpu().numpy()).astype(np.float32)   # 2^-128 and 6 * 2^127 included
    assert np.array_equal(out.cpu().numpy(), want, equal_nan=True)


def test_ranges_and_pages_out_of_bounds_leave_their_sequence():
    rng = np.random.default_rng(5)
    H, N, P, R = 2, 16, 16, 2
    pool = Pool([[]] * 5, H, N, P, R, "f32", rng, room=4)
    pool.table[3, 1] = pool.pages.shape[0]        # no such page: sequence 3 is not moved at all
    before = pool.pages.clone()
    dH, want = cast(rng.standard_normal((5, H, 3, N, P)), "f32")
    #                                            past the table, more than dH has, negative, bad page, good
    first, count = ints(2, 0, -1, 0, 1), ints(3, 4, 2, 3, 3)
    dart.dart_cache_write_paged(dH, first, count, pool.pages, pool.table)
    with pytest.raises(dart.DartError):
        dart.dart_sync_status()
    for m in range(1, 4):
        before[pool.table_np[4, m // R], :, m % R] = dH[4, :, m - 1]
    assert torch.equal(before.view(torch.int32), pool.pages.view(torch.int32))
    dart.dart_sync_status()                        # the error is reported once


# ---------------------------------------------------------------- recurrence
def extend_inputs(rng, lens, H, G, N, P, dtype, trailing=0):
    T = sum(lens) + trailing
    x, x64 = cast(rng.standard_normal((T, H, P)), dtype)
    Bm, B64 = cast(rng.standard_normal((T, G, N)) / np.sqrt(N), dtype)
    Cm, C64 = cast(rng.standard_normal((T, G, N)) / np.sqrt(N), dtype)
    dt, dt64 = cast(np.exp(rng.uniform(np.log(1e-3), np.log(1e-1), (T, H))), "f32")
    A, A64 = cast(-np.exp(rng.uniform(0, np.log(16), H)), "f32")
    return (x, dt, A, Bm, Cm), (x64, dt64, A64, B64, C64)


def states(rng, B, H, N, P):
    s, s64 = cast(rng.standard_normal((B, H, N, P)) / np.sqrt(N), "f32")
    c, c64 = cast(rng.standard_normal((B, H, N, P)) / np.sqrt(N), "f32")
    return s, c, s64, c64


def check_memory(got, want, cache, scales=None):
    """A memory rounded to the cache's type, against the float64 one it was computed for."""
    if cache == "f32":
        assert rel_err(got, want) <= TOL
    elif cache == "bf16":
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + TOL * np.abs(want).max()).all()
    else:
        # half a step of the code, whose scale is the least that holds the block's largest value
        N = want.shape[-2]
        unit = 2.0 ** (np.repeat(np.moveaxis(scales, -1, -2), 32, -2).astype(float) - 127)
        block = np.abs(want).reshape(*want.shape[:-2], N // 32, 32, -1).max(-2)
        low = unit.reshape(*want.shape[:-2], N // 32, 32, -1)[..., 0, :]
        assert (block <= 6 * low * (1 + TOL)).all() and (block > 3 * low * (1 - TOL)).all()
        a = np.abs(got) / unit
        step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
        assert (np.abs(got - want) <= step * unit / 2 + TOL * np.abs(want).max()).all()


@pytest.mark.parametrize("N, P, dtype, cache, H, G", [(128, 64, "bf16", "bf16", 4, 1), (128, 64, "bf16", "mxfp4", 2, 2),
                                                      (128, 64, "f32", "f32", 2, 1), (64, 64, "bf16", "bf16", 4, 2),
                                                      (64, 64, "f32", "mxfp4", 2, 1), (16, 16, "f32", "f32", 3, 3),
                                                      (16, 16, "bf16", "bf16", 2, 1)])
@pytest.mark.parametrize("lens, pos, S, R", [([1, 1, 1], [0, 7, 3], 8, 2), ([5, 0, 17, 2], [6, 7, 3, 6], 8, 3),
                                             ([33, 64, 1], [40, 0, 63], 64, 1), ([80], [250], 256, 4), ([3, 4], [0, 0], 1, 5)])
def test_extend(N, P, dtype, cache, H, G, lens, pos, S, R):
    rng = np.random.default_rng(sum(lens) + N)
    B = len(lens)
    n = [int(v) for v in rng.integers(0, 4, B)]
    have = memories_of(rng, n, H, N, P, cache)
    pool = Pool(have, H, N, P, R, cache, rng, room=max((p + t) // S for p, t in zip(pos, lens)))
    args, args64 = extend_inputs(rng, lens, H, G, N, P, dtype, trailing=3)
    s, c, s64, c64 = states(rng, B, H, N, P)
    y = torch.full((sum(lens) + 3, H, P), 9.0, device="cuda")
    seen = torch.full((sum(lens) + 3,), 99, dtype=torch.int32, device="cuda")
    before = (s.clone(), c.clone())
    got = dart.dart_ssd_extend(*args, cumulative(lens), s, c, pool.pages, pool.table, ints(*n), ints(*pos), S, scales=pool.scales,
                               state_out=torch.empty_like(s), dH_cur_out=torch.empty_like(c), y=y, mem_count=seen)
    dart.dart_sync_status()
    yr, sr, cr, nr, pr, counts, app = ref.extend(*args64, lens, s64, c64, n, pos, S)
    T = sum(lens)
    assert rel_err(y[:T], yr[:T]) <= TOL and (y[T:] == 9.0).all()
    assert rel_err(got["state"], sr) <= TOL and rel_err(got["dH_cur"], cr) <= TOL
    assert got["nchunks"].tolist() == nr and got["pos"].tolist() == pr
    assert seen.tolist() == counts + [99] * 3
    assert torch.equal(s, before[0]) and torch.equal(c, before[1])     # the old state is kept
    for b in range(B):
        for m, mem in enumerate(have[b]):
            assert np.array_equal(pool.memory(b, m), mem)              # the memories that were there too
        for j, mem in enumerate(app[b]):
            m = n[b] + j
            page, slot = pool.table_np[b, m // R], m % R
            check_memory(pool.memory(b, m), mem, cache, None if pool.scales is None else pool.scales[page, :, slot].cpu().numpy())
    # the same in place, bit for bit
    again = dart.dart_ssd_extend(*args, cumulative(lens), s, c, pool.pages, pool.table, ints(*n), ints(*pos), S, scales=pool.scales)
    dart.dart_sync_status()
    assert again["state"] is s and torch.equal(s, got["state"]) and torch.equal(c, got["dH_cur"])
    assert torch.equal(again["y"][:T], y[:T])


@pytest.mark.parametrize("N, H, G", [(128, 32, 1), (128, 2, 2), (64, 40, 8), (64, 1, 1)])
@pytest.mark.parametrize("cache", ["bf16", "mxfp4"])
@pytest.mark.parametrize("lens, pos, S", [([70, 0, 130, 5], [5, 1, 31, 30], 32), ([64, 65, 1], [0, 0, 99], 100), ([200], [250], 256)])
def test_extend_of_long_runs(N, H, G, cache, lens, pos, S):
    """Blocks of 64 tokens, full, partial and cut by the ends of chunks; some tokens forget nearly everything (dt A down
    to -80), others hardly anything.  float32 sums of up to 200 terms and differences of sums of logarithms: TOL."""
    rng = np.random.default_rng(sum(lens) + N + H)
    B, P = len(lens), 64
    n = [1] * B
    have = memories_of(rng, n, H, N, P, cache)
    pool = Pool(have, H, N, P, 3, cache, rng, room=max((p + t) // S for p, t in zip(pos, lens)))
    args, args64 = extend_inputs(rng, lens, H, G, N, P, "bf16", trailing=2)
    dt64 = args64[1] * np.where(rng.uniform(size=args64[1].shape) < 0.03, 50.0, 1.0)
    dt, dt64 = cast(dt64, "f32")
    args, args64 = (args[0], dt, *args[2:]), (args64[0], dt64, *args64[2:])
    s, c, s64, c64 = states(rng, B, H, N, P)
    y = torch.full((sum(lens) + 2, H, P), 9.0, device="cuda")
    call = lambda so, co, to: dart.dart_ssd_extend(*args, cumulative(lens), s, c, pool.pages, pool.table, ints(*n), ints(*pos), S,
                                                   scales=pool.scales, state_out=so, dH_cur_out=co, y=to)
    got = call(torch.empty_like(s), torch.empty_like(c), y)
    dart.dart_sync_status()
    yr, sr, cr, nr, pr, counts, app = ref.extend(*args64, lens, s64, c64, n, pos, S)
    T = sum(lens)
    assert rel_err(y[:T], yr[:T]) <= TOL and (y[T:] == 9.0).all()
    assert rel_err(got["state"], sr) <= TOL and rel_err(got["dH_cur"], cr) <= TOL
    assert got["nchunks"].tolist() == nr and got["pos"].tolist() == pr and got["mem_count"][:T].tolist() == counts
    for b in range(B):
        assert np.array_equal(pool.memory(b, 0), have[b][0])
        for j, mem in enumerate(app[b]):
            page, slot = pool.table_np[b, (1 + j) // 3], (1 + j) % 3
            check_memory(pool.memory(b, 1 + j), mem, cache, None if pool.scales is None else pool.scales[page, :, slot].cpu().numpy())
    again = call(s, c, torch.zeros_like(y))         # in place, and the same bits
    dart.dart_sync_status()
    assert torch.equal(again["y"][:T], y[:T]) and torch.equal(s, got["state"]) and torch.equal(c, got["dH_cur"])


def test_extend_leaves_what_it_cannot_do():
    """Full tables, bad pages and bad counters: the sequence keeps its state and counters, its tokens are marked."""
    rng = np.random.default_rng(6)
    H, N, P, S, lens = 2, 16, 16, 4, [3, 5, 2, 2, 6, 3]
    pool = Pool([[]] * 6, H, N, P, 1, "f32", rng, room=3)
    n, pos = [3, 0, -1, 0, 1, 0], [1, 2, 0, 4, 1, 2]    # no room; bad page; n < 0; pos = S; good; good
    pool.table[1, 0] = -5
    args, args64 = extend_inputs(rng, lens, H, 1, N, P, "f32")
    s, c, s64, c64 = states(rng, 6, H, N, P)
    pages = pool.pages.clone()
    y = torch.full((sum(lens), H, P), 9.0, device="cuda")
    got = dart.dart_ssd_extend(*args, cumulative(lens), s.clone(), c.clone(), pool.pages, pool.table, ints(*n), ints(*pos), S, y=y)
    with pytest.raises(dart.DartError) as e:
        dart.dart_sync_status()
    assert e.value.status == dart.DART_ERR_DEVICE
    good = [0, 0, 0, 0, 6, 3]
    starts = np.concatenate([[0], np.cumsum(lens)])
    yr, sr, cr, nr, pr, counts, app = ref.extend(*[np.concatenate([v[starts[4]:]]) if v.ndim > 1 else v for v in args64], good, s64, c64,
                                                 n, pos, S)
    assert (y[:starts[4]] == 9.0).all() and rel_err(y[starts[4]:], yr) <= TOL
    assert got["mem_count"].tolist() == [-1] * int(starts[4]) + counts
    assert got["nchunks"].tolist() == nr and got["pos"].tolist() == pr
    assert torch.equal(got["state"][:4], s[:4]) and torch.equal(got["dH_cur"][:4], c[:4])
    assert rel_err(got["state"], sr) <= TOL
    for b in (4, 5):
        for j, mem in enumerate(app[b]):
            m = n[b] + j
            assert rel_err(pool.memory(b, m), mem) <= TOL
            pages[pool.table_np[b, m]] = pool.pages[pool.table_np[b, m]]
    assert torch.equal(pages.view(torch.int32), pool.pages.view(torch.int32))


# ----------------------------------------------------------------- attention
def attention_inputs(rng, T, H, G, N, P, dtype, sharp=1.0):
    Q, Q64 = cast(rng.standard_normal((T, H, N)) * sharp, dtype)
    E, E64 = cast(rng.standard_normal((T, H, P)) / np.sqrt(P), dtype)
    C, C64 = cast(rng.standard_normal((T, G, N)) / np.sqrt(N), dtype)
    return (Q, E, C), (Q64, E64, C64)


SHAPES = [(128, 64, "bf16", "bf16", 4, 1), (128, 64, "bf16", "mxfp4", 2, 2), (128, 64, "f32", "mxfp4", 2, 1),
          (128, 64, "f32", "f32", 2, 1), (64, 64, "bf16", "bf16", 4, 2), (64, 64, "f32", "f32", 2, 2), (64, 64, "bf16", "mxfp4", 4, 4),
          (64, 64, "f32", "mxfp4", 1, 1), (16, 16, "f32", "f32", 3, 3), (16, 16, "bf16", "bf16", 2, 1)]


@pytest.mark.parametrize("N, P, dtype, cache, H, G", SHAPES)
@pytest.mark.parametrize("lens, mems, R", [([1], [0], 1), ([1], [1], 4), ([1, 1, 1, 1, 1], [5, 0, 33, 1, 16], 16),
                                           ([2, 0, 9, 1, 70], [3, 4, 17, 150, 29], 7), ([130, 3], [40, 5], 1)])
def test_attention(N, P, dtype, cache, H, G, lens, mems, R):
    """Counts within a sequence differ from row to row, none and rows left out among them; what follows a sequence's
    last memory in its page is NaN, and so is the rest of the pool."""
    rng = np.random.default_rng(sum(lens) + sum(mems) + N)
    memories = memories_of(rng, mems, H, N, P, cache, scale=0.5)
    pool = Pool(memories, H, N, P, R, cache, rng)
    T = sum(lens)
    args, args64 = attention_inputs(rng, T + 2, H, G, N, P, dtype)
    counts = [int(rng.integers(max(0, m - 3), m + 1)) for k, m in zip(lens, mems) for _ in range(k)]
    if T > 20:
        counts[1], counts[4], counts[-1] = 0, -1, mems[-1]
    y, y64 = cast(rng.standard_normal((T + 2, H, P)) * 0.1, "f32")
    o = ref.sma(*[v[:T] for v in args64], lens, memories, counts)
    want = np.where((np.array(counts) >= 0)[:, None, None], y64[:T] + 0.7 * o, 5.0)
    out = torch.full_like(y, 5.0)
    seen = ints(*counts, 1000, -7)                       # rows that no sequence owns are not looked at
    dart.dart_sma_paged(*args, cumulative(lens), pool.pages, pool.table, seen, 0.7, y, scales=pool.scales, out=out)
    dart.dart_sync_status()
    assert rel_err(out[:T], want) <= TOL and (out[T:] == 5.0).all()
    # without y_ssd: the readout itself
    out2 = torch.full_like(y, 5.0)
    dart.dart_sma_paged(*args, cumulative(lens), pool.pages, pool.table, seen, 0.7, scales=pool.scales, out=out2)
    assert rel_err(out2[:T], np.where((np.array(counts) >= 0)[:, None, None], o, 5.0)) <= TOL
    # in place over y_ssd, and the same bits every time
    z = y.clone()
    z[torch.tensor(counts + [0, 0], device="cuda") < 0] = 5.0
    z[T:] = 5.0
    dart.dart_sma_paged(*args, cumulative(lens), pool.pages, pool.table, seen, 0.7, z, scales=pool.scales, out=z)
    dart.dart_sync_status()
    assert torch.equal(z, out)


@pytest.mark.parametrize("N, P, dtype, cache, H, G", SHAPES)
def test_attention_over_many_memories_is_shared_by_blocks(N, P, dtype, cache, H, G):
    """Few rows, many memories: the runs of several blocks meet in one row.  One score stands out by far."""
    rng = np.random.default_rng(N + H)
    lens, mems = [1, 4], [901, 400]
    memories = memories_of(rng, mems, H, N, P, cache, scale=0.5)
    pool = Pool(memories, H, N, P, 16, cache, rng)
    args, args64 = attention_inputs(rng, 5, H, G, N, P, dtype, sharp=4.0)
    counts = [901, 400, 399, 17, 400]
    out = dart.dart_sma_paged(*args, cumulative(lens), pool.pages, pool.table, ints(*counts), 1.0, scales=pool.scales)
    dart.dart_sync_status()
    assert rel_err(out, ref.sma(*args64, lens, memories, counts)) <= 2 * TOL    # scores are up to 4 times those of TOL, mostly half that


@pytest.mark.parametrize("N, P, dtype, cache, H, G", SHAPES)
def test_attention_rows_with_bad_pages_or_counts_are_left(N, P, dtype, cache, H, G):
    rng = np.random.default_rng(8)
    lens, mems, R = [3, 2, 1], [9, 6, 4], 2
    memories = memories_of(rng, mems, H, N, P, cache, scale=0.5)
    pool = Pool(memories, H, N, P, R, cache, rng)
    args, args64 = attention_inputs(rng, 6, H, G, N, P, dtype)
    counts = [9, 4, 5, 6, 2, 4]
    o = ref.sma(*args64, lens, memories, counts)
    pool.table[0, 2] = pool.pages.shape[0] + 3           # memories 4 and 5 of sequence 0: rows that see them are left
    seen = ints(9, 4, 5, 99, 2, 4)                       # 99: more than the table holds
    out = torch.full((6, H, P), 5.0, device="cuda")
    dart.dart_sma_paged(*args, cumulative(lens), pool.pages, pool.table, seen, 1.0, scales=pool.scales, out=out)
    with pytest.raises(dart.DartError):
        dart.dart_sync_status()
    left = [0, 2, 3]
    assert (out[left] == 5.0).all()
    done = [1, 4, 5]
    assert rel_err(out[done], o[done]) <= TOL


@pytest.mark.parametrize("N, P, dtype, cache, H, G", [v for v in SHAPES if v[3] != "f32" and v[1] == 64])
@pytest.mark.parametrize("lens, mems, R", [([20, 33], [6, 5], 4), ([64, 0, 128, 1, 200], [9, 3, 2, 5, 13], 3), ([257], [50], 16),
                                           ([300, 100, 260], [4, 1, 7], 2), ([129, 128], [0, 21], 5)])
def test_attention_of_long_runs(N, P, dtype, cache, H, G, lens, mems, R):
    """Runs that fill tiles of 128 and 256 rows and end inside them; a page of the last sequence is missing, and rows
    whose count reaches it are left as they are, and so are those marked with -1."""
    rng = np.random.default_rng(sum(lens) + sum(mems) + N)
    memories = memories_of(rng, mems, H, N, P, cache, scale=0.5)
    pool = Pool(memories, H, N, P, R, cache, rng)
    T = sum(lens)
    args, args64 = attention_inputs(rng, T + 3, H, G, N, P, dtype)
    counts = [min(m, max(0, m - 2 + i * 3 // k)) for k, m in zip(lens, mems) for i in range(k)]
    counts[3] = 0
    o = ref.sma(*[v[:T] for v in args64], lens, memories, counts)
    seen = np.array(counts)
    bad = mems[-1] > R
    if bad:
        pool.table[len(lens) - 1, (mems[-1] - 1) // R] = -1
        last = np.arange(T) >= T - lens[-1]
        left = last & (seen > (mems[-1] - 1) // R * R)
    else:
        left = np.zeros(T, bool)
    seen[T // 2] = -1
    left[T // 2] = True
    y, y64 = cast(rng.standard_normal((T + 3, H, P)) * 0.1, "f32")
    want = np.where(left[:, None, None], 5.0, y64[:T] + 0.7 * o)
    out = torch.full_like(y, 5.0)
    call = lambda to: dart.dart_sma_paged(*args, cumulative(lens), pool.pages, pool.table, ints(*seen.tolist(), 9, 9, 9), 0.7, y,
                                          scales=pool.scales, out=to)
    call(out)
    if bad:
        with pytest.raises(dart.DartError):
            dart.dart_sync_status()
    else:
        dart.dart_sync_status()
    assert rel_err(out[:T], want) <= TOL and (out[T:] == 5.0).all()
    again = torch.full_like(y, 5.0)
    call(again)
    assert torch.equal(again, out)
    if bad:
        with pytest.raises(dart.DartError):
            dart.dart_sync_status()


@pytest.mark.parametrize("N, P, dtype, cache, H, G", [v for v in SHAPES if v[3] == "bf16" and v[1] == 64])
@pytest.mark.parametrize("lens", [[40], [150]])
def test_long_runs_over_many_memories_are_shared_by_blocks(N, P, dtype, cache, H, G, lens):
    rng = np.random.default_rng(N + H + lens[0])
    memories = memories_of(rng, [700], H, N, P, cache, scale=0.5)
    pool = Pool(memories, H, N, P, 16, cache, rng)
    args, args64 = attention_inputs(rng, lens[0], H, G, N, P, dtype)
    counts = [700 - (i % 5) for i in range(lens[0])]
    counts[1], counts[2] = 3, 0
    out = dart.dart_sma_paged(*args, cumulative(lens), pool.pages, pool.table, ints(*counts), 1.0, scales=pool.scales)
    dart.dart_sync_status()
    assert rel_err(out, ref.sma(*args64, lens, memories, counts)) <= TOL


@pytest.mark.parametrize("N, P, dtype, cache, H, G", SHAPES)
@pytest.mark.parametrize("lens", [[4], [40], [150]])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(N, P, dtype, cache, H, G, lens):
    """The last two memories hold NaN (a block of them in 4-bit pages) and, where the format has it, an infinity; rows
    that do not see them are as if they were not there, rows that do are NaN."""
    rng = np.random.default_rng(N + lens[0])
    memories = memories_of(rng, [12], H, N, P, cache, scale=0.5)
    pool = Pool(memories, H, N, P, 5, cache, rng)
    page, slot = pool.table_np[0, 10 // 5], 10 % 5
    nan, inf = (pool.pages[page, :, slot + i] for i in range(2))
    if cache == "mxfp4":
        pool.scales[page, :, slot, 7, 1] = 255
        pool.scales[page, :, slot + 1, 9, 0] = 255
    else:
        nan[:, N - 1, P - 1] = float("nan")
        inf[:, 3, 2] = float("inf")
    args, args64 = attention_inputs(rng, lens[0], H, G, N, P, dtype)
    counts = [10 + (i % 4 == 1) + 2 * (i % 4 == 3) for i in range(lens[0])]
    out = dart.dart_sma_paged(*args, cumulative(lens), pool.pages, pool.table, ints(*counts), 1.0, scales=pool.scales)
    dart.dart_sync_status()
    fine = np.array(counts) == 10
    want = ref.sma(*args64, lens, memories, [10] * lens[0])
    assert rel_err(out[fine], want[fine]) <= TOL
    assert torch.isnan(out[~fine]).all()


@pytest.mark.parametrize("N, P, dtype, cache, H, G", SHAPES)
@pytest.mark.parametrize("lens", [[3], [33], [140]])
def test_a_bad_page_in_a_shared_item(N, P, dtype, cache, H, G, lens):
    """An item over many blocks whose 15th page of 20 is missing: rows that see it are left, whoever finds it."""
    rng = np.random.default_rng(H + lens[0])
    memories = memories_of(rng, [320], H, N, P, cache, scale=0.5)
    pool = Pool(memories, H, N, P, 16, cache, rng)
    args, args64 = attention_inputs(rng, lens[0], H, G, N, P, dtype)
    counts = [(320, 224, 225)[i % 3] for i in range(lens[0])]
    pool.table[0, 14] = pool.pages.shape[0]
    out = torch.full((lens[0], H, P), 5.0, device="cuda")
    dart.dart_sma_paged(*args, cumulative(lens), pool.pages, pool.table, ints(*counts), 1.0, scales=pool.scales, out=out)
    with pytest.raises(dart.DartError):
        dart.dart_sync_status()
    done = np.array(counts) == 224
    want = ref.sma(*args64, lens, memories, [224] * lens[0])
    assert rel_err(out[done], want[done]) <= TOL and (out[~done] == 5.0).all()


@pytest.mark.parametrize("N, P, dtype, cache, H, G", SHAPES)
def test_many_sequences(N, P, dtype, cache, H, G):
    """More sequences than a block has threads, some without tokens, some without memories, most with a few of both."""
    rng = np.random.default_rng(21)
    B = 900
    lens = [int(v) for v in rng.integers(0, 3, B)]
    mems = [int(v) for v in rng.integers(0, 3, B)]
    one = memories_of(rng, [4], H, N, P, cache, scale=0.5)[0]
    pool = Pool([one], H, N, P, 2, cache, rng)
    pool.table = pool.table.expand(B, 2).contiguous()             # all read the same pages
    T = sum(lens)
    args, args64 = attention_inputs(rng, T, H, G, N, P, dtype)
    counts = [mems[b] for b in range(B) for _ in range(lens[b])]
    out = dart.dart_sma_paged(*args, cumulative(lens), pool.pages, pool.table, ints(*counts), 1.0, scales=pool.scales)
    dart.dart_sync_status()
    assert rel_err(out, ref.sma(*args64, lens, [one] * B, counts)) <= TOL


def test_calls_without_tokens():
    rng = np.random.default_rng(22)
    H, N, P = 2, 64, 64
    pool = Pool(memories_of(rng, [2, 1], H, N, P, "bf16"), H, N, P, 2, "bf16", rng)
    args, _ = extend_inputs(rng, [0, 0], H, 1, N, P, "bf16")
    s, c, s64, c64 = states(rng, 2, H, N, P)
    s2, c2 = torch.zeros_like(s), torch.zeros_like(c)
    got = dart.dart_ssd_extend(*args, ints(0, 0, 0), s, c, pool.pages, pool.table, ints(2, 1), ints(3, 0), 4, state_out=s2, dH_cur_out=c2)
    att, _ = attention_inputs(rng, 0, H, 1, N, P, "bf16")
    out = dart.dart_sma_paged(*att, ints(0, 0, 0), pool.pages, pool.table, got["mem_count"], 1.0)
    dart.dart_sync_status()
    assert out.shape == (0, H, P) and torch.equal(s2, s) and torch.equal(c2, c)
    assert got["nchunks"].tolist() == [2, 1] and got["pos"].tolist() == [3, 0]


def test_views_and_host_tensors_as_inputs():
    """Token tensors that are slices of wider ones, or on the host, are taken as what they hold."""
    rng = np.random.default_rng(23)
    H, N, P, lens, mems = 2, 128, 64, [3, 20], [4, 9]
    memories = memories_of(rng, mems, H, N, P, "bf16", scale=0.5)
    pool = Pool(memories, H, N, P, 4, "bf16", rng)
    (Q, E, C), args64 = attention_inputs(rng, 23, H, 1, N, P, "bf16")
    counts = [mems[0]] * 3 + [mems[1]] * 20
    wide = torch.zeros((23, H, 2 * N), dtype=torch.bfloat16, device="cuda")
    wide[..., N:] = Q
    plain = dart.dart_sma_paged(Q, E, C, cumulative(lens), pool.pages, pool.table, ints(*counts), 1.0)
    view = dart.dart_sma_paged(wide[..., N:], E.transpose(0, 1).contiguous().transpose(0, 1), C[:, 0], cumulative(lens), pool.pages,
                               pool.table, ints(*counts), 1.0)
    host = dart.dart_sma_paged(Q.cpu(), E.cpu(), C.cpu(), cumulative(lens), pool.pages, pool.table, ints(*counts), 1.0)
    dart.dart_sync_status()
    assert torch.equal(view, plain) and torch.equal(host, plain)


def test_two_calls_at_once():
    """Two streams, each with its own inputs and workspace, many times over: the same bits as one after the other."""
    rng = np.random.default_rng(24)
    H, N, P = 4, 128, 64
    work = []
    for lens, mems, cache in (([1] * 20, [40] * 20, "bf16"), ([3] * 15, [60] * 15, "mxfp4"), ([100, 60], [30, 50], "bf16")):
        memories = memories_of(rng, [max(mems)], H, N, P, cache, scale=0.5)
        pool = Pool(memories, H, N, P, 8, cache, rng)
        pool.table = pool.table.expand(len(lens), pool.table.shape[1]).contiguous()
        args, _ = attention_inputs(rng, sum(lens), H, 1, N, P, "bf16")
        counts = ints(*[m for k, m in zip(lens, mems) for _ in range(k)])
        cu = cumulative(lens)
        work.append(lambda a=args, cu=cu, p=pool, c=counts: dart.dart_sma_paged(*a, cu, p.pages, p.table, c, 1.0, scales=p.scales))
    want = [f() for f in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(20):
        got = []
        for f, st in zip(work, streams):
            with torch.cuda.stream(st):
                got.append(f())
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    dart.dart_sync_status()


def test_a_shared_page_is_read_by_two_sequences():
    rng = np.random.default_rng(9)
    H, N, P, R = 2, 128, 64, 4
    memories = memories_of(rng, [4, 0], H, N, P, "bf16", scale=0.5)
    pool = Pool(memories, H, N, P, R, "bf16", rng)
    pool.table[1, 0] = pool.table[0, 0]
    args, args64 = attention_inputs(rng, 3, H, 1, N, P, "bf16")
    out = dart.dart_sma_paged(*args, cumulative([1, 2]), pool.pages, pool.table, ints(4, 3, 2), 1.0)
    dart.dart_sync_status()
    assert rel_err(out, ref.sma(*args64, [1, 2], [memories[0], memories[0]], [4, 3, 2])) <= TOL


@pytest.mark.parametrize("cache", ["bf16", "mxfp4"])
def test_pages_beyond_32_bit_offsets(cache):
    """The last pages of a pool of more than 2^32 bytes (2^31 elements and over)."""
    H, N, P, R = 32, 128, 64, 16
    one = H * R * N * P * (2 if cache == "bf16" else 0.5)
    npages = int(2 ** 32 // one) + 40
    if cache == "bf16":
        pages, scales = torch.empty((npages, H, R, N, P), dtype=torch.bfloat16, device="cuda"), None
    else:
        pages = torch.empty((npages, H, R, P, N // 2), dtype=torch.uint8, device="cuda")
        scales = torch.empty((npages, H, R, P, N // 32), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(11)
    memories = memories_of(rng, [20], H, N, P, cache, scale=0.5)
    dH = torch.from_numpy(np.moveaxis(memories[0], 0, 1)[None].copy()).bfloat16().cuda()
    table = ints(npages - 1, npages - 2).reshape(1, 2)
    dart.dart_cache_write_paged(dH, ints(0), ints(20), pages, table, scales=scales)
    out = torch.zeros_like(dH)
    dart.dart_cache_read_paged(pages, table, ints(0), ints(20), out=out, scales=scales)
    args, args64 = attention_inputs(rng, 2, H, 1, N, P, "bf16")
    o = dart.dart_sma_paged(*args, ints(0, 2), pages, table, ints(20, 19), 1.0, scales=scales)
    dart.dart_sync_status()
    assert torch.equal(out, dH)
    assert rel_err(o, ref.sma(*args64, [2], memories, [20, 19])) <= TOL


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("cache", ["bf16", "mxfp4"])
def test_prompt_then_pieces_then_tokens_is_the_whole_layer(cache):
    """Prefill by the chunked scan, handed over to pages, then a piece of the prompt, drafts and single tokens; against
    the recurrence and the attention over the memories that the pages hold."""
    rng = np.random.default_rng(12)
    H, G, N, P, S, R = 4, 1, 128, 64, 256, 2
    L0, pieces = [256 * 2 + 100, 256 + 7], [[300, 1], [5, 3], [1, 1], [0, 6]]
    more = [sum(p[b] for p in pieces) for b in range(2)]
    pool = Pool([[], []], H, N, P, R, cache, rng, room=5)
    g = 0.6
    drawn = [(extend_inputs(rng, [L0[b] + more[b]], H, G, N, P, "bf16"), attention_inputs(rng, L0[b] + more[b], H, G, N, P, "bf16"))
             for b in range(2)]
    all_args = [(e[0], q[0], e[1], q[1]) for e, q in drawn]
    A, A64 = all_args[0][0][2], all_args[0][2][2]        # one A for both
    state, cur, n, pos = [], [], [], []
    for b in range(2):
        x, dt, _, Bm, Cm = (v[None, :L0[b]] if v.dim() > 1 else v for v in all_args[b][0])
        _, dH, st = dart.dart_ssd_chunk_scan(x, dt, A, Bm, Cm, S)
        done = L0[b] // S
        dart.dart_cache_write_paged(dH, ints(0), ints(done), pool.pages, pool.table[b:b + 1], scales=pool.scales)
        state.append(st[0, :, -1])
        cur.append(dH[0, :, -1].float())
        n.append(done)
        pos.append(L0[b] % S)
    s, c = torch.stack(state).contiguous(), torch.stack(cur).contiguous()
    s64, c64 = f64(s), f64(c)
    nt, pt, at = ints(*n), ints(*pos), list(L0)
    for lens in pieces:
        rows = [slice(at[b], at[b] + lens[b]) for b in range(2)]
        cat = lambda k, i: torch.cat([all_args[b][k][i][rows[b]] for b in range(2)]).contiguous()
        cat64 = lambda k, i: np.concatenate([all_args[b][k][i][rows[b]] for b in range(2)])
        res = dart.layer_extend(cat(0, 0), cat(0, 1), A, cat(0, 3), cat(0, 4), cat(1, 0), cat(1, 1), g, cumulative(lens), s, c,
                                pool.pages, pool.table, nt, pt, S, scales=pool.scales)
        dart.dart_sync_status()
        yr, s64, c64, n2, p2, counts, app = ref.extend(cat64(2, 0), cat64(2, 1), A64, cat64(2, 3), cat64(2, 4), lens, s64, c64, n, pos, S)
        held = [np.stack([pool.memory(b, m) for m in range(n2[b])]) for b in range(2)]
        o = ref.sma(cat64(3, 0), cat64(3, 1), cat64(2, 4), lens, held, counts)
        assert rel_err(res["y"], yr + g * o) <= 2 * TOL          # two operators' errors; runs of 300 tokens
        assert rel_err(res["state"], s64) <= 2 * TOL and rel_err(res["dH_cur"], c64) <= 2 * TOL
        assert res["nchunks"].tolist() == n2 and res["pos"].tolist() == p2 and res["mem_count"].tolist() == counts
        for b in range(2):
            for j, mem in enumerate(app[b]):
                m = n[b] + j
                page, slot = pool.table_np[b, m // R], m % R
                check_memory(pool.memory(b, m), mem, cache, None if pool.scales is None else pool.scales[page, :, slot].cpu().numpy())
        n, pos, nt, pt = n2, p2, res["nchunks"], res["pos"]
        at = [at[b] + lens[b] for b in range(2)]
    assert n == [3, 1] and max(n) > 2


def test_single_tokens_agree_with_the_dense_decode_step():
    shape = synth.DecodeShape(4, 4, 64, 128, 4, 5, 8, 9, "bf16")
    init = synth.decode_initial(shape, seed=2)
    init["nchunks"] = torch.tensor([5, 0, 3, 1], dtype=torch.int32)
    init["pos"] = torch.tensor([0, 3, 1, 2], dtype=torch.int32)
    d = {k: v.cuda() for k, v in init.items()}
    A = synth.decode_A(shape, 2).cuda()
    rng = np.random.default_rng(1)
    have = [[f64(d["cache"][b, :, m]) for m in range(int(init["nchunks"][b]))] for b in range(4)]
    pool = Pool(have, 4, 128, 64, 3, "bf16", rng, room=3)
    s, c, n, pos = d["state"].clone(), d["dH_cur"].clone(), d["nchunks"].clone(), d["pos"].clone()
    for step in range(9):
        t = {k: v.cuda() for k, v in synth.decode_tokens(shape, step, 2).items()}
        y = dart.dart_decode_step(t["x"], t["dt"], A, t["Bm"], t["Cm"], t["Q"], t["E"], 0.5, d["state"], d["dH_cur"], d["cache"],
                                  d["nchunks"], d["pos"], 4)
        res = dart.layer_extend(t["x"], t["dt"], A, t["Bm"], t["Cm"], t["Q"], t["E"], 0.5, cumulative([1] * 4), s, c, pool.pages,
                                pool.table, n, pos, 4)
        dart.dart_sync_status()
        n, pos = res["nchunks"], res["pos"]
        assert rel_err(res["y"], f64(y)) <= TOL
        assert torch.equal(n, d["nchunks"]) and torch.equal(pos, d["pos"])
        assert rel_err(s, f64(d["state"])) <= TOL
    for b in range(4):
        for m in range(int(n[b])):
            # the same float32 memory up to its last bits, rounded to bfloat16 twice
            np.testing.assert_allclose(pool.memory(b, m), f64(d["cache"][b, :, m]), rtol=2.0 ** -7, atol=1e-6)


def test_drafts_are_taken_back():
    """A run of drafts into a state of its own, then the accepted ones from the old state: as if only they had come."""
    rng = np.random.default_rng(13)
    H, N, P, S, lens, taken = 2, 64, 64, 4, [6, 5, 3], [2, 5, 0]
    pool = Pool([[], [], []], H, N, P, 2, "f32", rng, room=3)
    args, args64 = extend_inputs(rng, lens, H, 1, N, P, "f32")
    s, c, s64, c64 = states(rng, 3, H, N, P)
    n, pos = ints(0, 1, 0), ints(3, 0, 2)
    dart.dart_ssd_extend(*args, cumulative(lens), s, c, pool.pages, pool.table, n, pos, S, state_out=torch.empty_like(s),
                         dH_cur_out=torch.empty_like(c))
    starts = np.concatenate([[0], np.cumsum(lens)])
    keep = np.concatenate([np.arange(starts[b], starts[b] + taken[b]) for b in range(3)])
    kept = [v[torch.from_numpy(keep).cuda()].contiguous() if v.dim() > 1 else v for v in args]
    got = dart.dart_ssd_extend(*kept, cumulative(taken), s, c, pool.pages, pool.table, n, pos, S)
    dart.dart_sync_status()
    yr, sr, cr, nr, pr, counts, app = ref.extend(*[v[keep] if v.ndim > 1 else v for v in args64], taken, s64, c64, [0, 1, 0], [3, 0, 2], S)
    assert rel_err(got["y"], yr) <= TOL and rel_err(s, sr) <= TOL and rel_err(c, cr) <= TOL
    assert got["nchunks"].tolist() == nr and got["pos"].tolist() == pr
    for b in range(3):
        for j, mem in enumerate(app[b]):
            assert rel_err(pool.memory(b, [0, 1, 0][b] + j), mem) <= TOL


# --------------------------------------------------- streams, graphs, devices
@pytest.mark.parametrize("cache", ["bf16", "mxfp4"])
def test_captured_and_replayed_with_other_inputs(cache):
    """Two graphs that run one after the other, each replayed on new token values; and the same on another stream."""
    rng = np.random.default_rng(14)
    H, N, P, S, R = 4, 128, 64, 8, 2
    mems = [5, 2, 0]
    memories = memories_of(rng, mems, H, N, P, cache, scale=0.5)
    pool = Pool(memories, H, N, P, R, cache, rng, room=3)
    s, c, s64, c64 = states(rng, 3, H, N, P)
    n, pos = ints(*mems), ints(0, 6, 3)
    sets = []
    for lens in ([1, 1, 1], [3, 4, 2]):
        args, _ = extend_inputs(rng, lens, H, 1, N, P, "bf16")
        att, _ = attention_inputs(rng, sum(lens), H, 1, N, P, "bf16")
        sets.append([lens, list(args), list(att), cumulative(lens), torch.empty_like(s), torch.empty_like(c)])

    def step(k):
        lens, a, q, cu, so, co = sets[k]
        return dart.layer_extend(*a, q[0], q[1], 0.5, cu, s, c, pool.pages, pool.table, n, pos, S, scales=pool.scales, state_out=so,
                                 dH_cur_out=co)

    for k in range(2):
        step(k)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(k))
        graphs.append(g)
    for trial in range(3):
        for k in range(2):
            lens, a, q, cu, so, co = sets[k]
            new, new64 = extend_inputs(rng, lens, H, 1, N, P, "bf16")
            att, att64 = attention_inputs(rng, sum(lens), H, 1, N, P, "bf16")
            for old, v in zip(a, new):
                old.copy_(v)
            for old, v in zip(q, att):
                old.copy_(v)
            graphs[k].replay()
            dart.dart_sync_status()
            yr, sr, cr, nr, pr, counts, app = ref.extend(*new64, lens, s64, c64, mems, [0, 6, 3], S)
            held = [[pool.memory(b, m) for m in range(nr[b])] for b in range(3)]
            held = [np.stack(v) if v else np.zeros((0, H, N, P)) for v in held]
            o = ref.sma(att64[0], att64[1], new64[4], lens, held, counts)
            assert rel_err(outs[k]["y"], yr + 0.5 * o) <= TOL
            assert rel_err(so, sr) <= TOL and outs[k]["nchunks"].tolist() == nr
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                other = step(k)
            side.synchronize()
            assert torch.equal(other["y"], outs[k]["y"])


def test_binding_refusals():
    rng = np.random.default_rng(15)
    H, N, P = 2, 128, 64
    pool = Pool(memories_of(rng, [2], H, N, P, "bf16"), H, N, P, 2, "bf16", rng)
    four = Pool(memories_of(rng, [2], H, N, P, "mxfp4"), H, N, P, 2, "mxfp4", rng)
    (Q, E, C), _ = attention_inputs(rng, 1, H, 1, N, P, "bf16")
    cu, seen = ints(0, 1), ints(2)
    ok = lambda **k: dart.dart_sma_paged(**{**dict(Q=Q, E=E, Cm=C, cu_tokens=cu, pages=pool.pages, table=pool.table, mem_count=seen,
                                                   g=1.0), **k})
    ok()
    for k in (dict(Q=Q.float(), E=E.float(), Cm=C.float()), dict(cu_tokens=cu.long()), dict(table=pool.table.long()),
              dict(mem_count=seen.float()), dict(pages=four.pages), dict(out=torch.empty((1, H, P), dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(TypeError):
            ok(**k)
    for k in (dict(cu_tokens=ints(0)), dict(mem_count=ints(2, 2)), dict(table=pool.table[:0]), dict(scales=four.scales),
              dict(pages=pool.pages[:, :1].contiguous()), dict(pages=pool.pages.transpose(3, 4)), dict(E=E[..., :32].contiguous()),
              dict(pages=four.pages, scales=four.scales[..., :2].contiguous()), dict(Cm=C[..., :64].contiguous()),
              dict(out=torch.empty((2, H, P), device="cuda")), dict(table=pool.table.cpu())):
        with pytest.raises(ValueError):
            ok(**k)
    with pytest.raises(dart.DartError):
        ok(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    dart.dart_sync_status()


def test_launch_count_grows_by_what_is_launched():
    rng = np.random.default_rng(16)
    pool = Pool(memories_of(rng, [2], 2, 128, 64, "bf16"), 2, 128, 64, 2, "bf16", rng)
    (Q, E, C), _ = attention_inputs(rng, 1, 2, 1, 128, 64, "bf16")
    before = dart.launch_count()
    dart.dart_sma_paged(Q, E, C, ints(0, 1), pool.pages, pool.table, ints(2), 1.0)
    assert dart.launch_count() == before + 2
