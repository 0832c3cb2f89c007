"""The paged 8-bit cache on the GPU against the plain 64-bit forms of tests/kv_reference.py.
Block assignment and the append (codes and scales) are compared exactly; the attention within
the bound that kv_reference.attention_tolerance derives from its roundings."""
import numpy as np
import pytest
import torch

from gated_linear_attention_liger_b200 import ops
from tests import kv_reference as ref
from tests.canary import Guarded, guarded_like

pytestmark = pytest.mark.gpu

E4M3, INT8 = torch.float8_e4m3fn, torch.int8
BF16, FP32 = torch.bfloat16, torch.float32


def i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


# ------------------------------------------------------------------ block assignment

def _state(rng, B, width, bs, lens, spare):
    """Tables, ring and span of a cache in use."""
    need = [-(-n // bs) for n in lens]
    n = sum(need) + spare
    perm = [int(x) for x in rng.permutation(n)]
    table, at = [], 0
    for k in need:
        table.append(perm[at:at + k] + [-1] * (width - k))
        at += k
    head = int(rng.integers(0, n))
    ring = [-7] * n
    for i, b in enumerate(perm[at:]):
        ring[(head + i) % n] = b
    return table, ring, [head, n - at]


def _check_assign(dev, new, lens, table, ring, span, bs, n_slots, in_place=False):
    t = [i32(x, dev) for x in (new, lens, table, ring, span)]
    kw = dict(seq_lens_out=t[1], free_span_out=t[4]) if in_place else {}
    slots, cu, lo, so = ops.kv_cache_assign(*t, bs, n_slots, **kw)
    table, ring = [list(r) for r in table], list(ring)
    want = ref.assign(list(new), list(lens), table, ring, list(span), bs, n_slots)
    got = (slots, cu, lo, so)
    for name, g, w in zip(("slots", "cu", "lens", "span"), got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), np.asarray(w, dtype=np.int32).reshape(g.shape), err_msg=name)
    np.testing.assert_array_equal(t[2].cpu().numpy(), np.asarray(table), err_msg="table")
    np.testing.assert_array_equal(t[3].cpu().numpy(), np.asarray(ring), err_msg="ring")


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("B", [1, 7, 64, 513])
def test_assign_grow_and_end(B, bs, cuda_device):
    rng = np.random.default_rng(100 * B + bs)
    width = 9
    lens = [int(x) for x in rng.integers(0, width * bs - 4, B)]
    new = [int(x) for x in rng.choice([-1, 0, 1, 2, 4], B)]
    _check_assign(cuda_device, new, lens, *_state(rng, B, width, bs, lens, 2 * B), bs, sum(max(x, 0) for x in new) + 3)


def test_assign_lengths_at_block_borders(cuda_device):
    rng = np.random.default_rng(1)
    lens = [0, 15, 16, 17, 31, 32, 33, 160, 159, 144]
    new = [0, 1, 1, 15, 1, 0, 100, 1, 1, 16]      # the eighth is full (its row has no block left)
    _check_assign(cuda_device, new, lens, *_state(rng, 10, 10, 16, lens, 20), 16, 140)


@pytest.mark.parametrize("spare", [0, 1, 3])
def test_assign_runs_out_of_blocks(spare, cuda_device):
    """The first that does not fit, and those behind it that need a block, get nothing."""
    rng = np.random.default_rng(2)
    lens = [16, 30, 5, 16, 0, 8]
    new = [1, 1, 1, 40, 1, 2]
    _check_assign(cuda_device, new, lens, *_state(rng, 6, 8, 16, lens, spare), 16, 60)


def test_assign_slot_map_too_short_and_none(cuda_device):
    rng = np.random.default_rng(3)
    lens, new = [3, 0, 20, 9], [4, 2, 10, 1]
    for n_slots in (0, 1, 6, 15, 16, 17):
        _check_assign(cuda_device, new, lens, *_state(rng, 4, 8, 16, lens, 9), 16, n_slots)


def test_assign_malformed_entries_stay_in_bounds(cuda_device):
    """Table entries that are no block give slots of -1; negative and overlong lengths are clamped."""
    dev = cuda_device
    table = [[5, -1, 99, 3], [2, 1, 0, 4]]
    slots, cu, lo, _ = ops.kv_cache_assign(i32([2, 1], dev), i32([15, -9], dev), i32(table, dev), i32([6, 7] + [0] * 6, dev),
                                           i32([0, 2], dev), 16, 4)
    assert slots.tolist() == [5 * 16 + 15, 6 * 16, 7 * 16, -1] and lo.tolist() == [17, 1]
    table = [[5, -1, 99, 3]]
    for n, want in ((16, -1), (33, -1), (48, 3 * 16)):
        got = ops.kv_cache_assign(i32([1], dev), i32([n], dev), i32([[5, -1, 99, 3]], dev), i32([3] + [0] * 7, dev),
                                  i32([0, 1], dev), 16, 1)
        if n % 16:
            assert got[0].tolist() == [want]
    got = ops.kv_cache_assign(i32([0], dev), i32([1 << 30], dev), i32(table, dev), i32([3] + [0] * 7, dev), i32([-4, 99], dev), 16, 1)
    assert got[2].tolist() == [64]


@pytest.mark.parametrize("B", [1, 40, 600])
def test_assign_many_slots(B, cuda_device):
    """Slot maps that many CTAs write, with the state advanced in place by a second launch."""
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 50, B)]
    new = [int(x) for x in rng.integers(0, 60000 // B, B)]
    new[B // 2] = -1 if B > 1 else new[0]
    width = -(-(50 + 60000 // B) // 16)
    st = _state(rng, B, width, 16, lens, B * width)
    _check_assign(cuda_device, new, lens, *st, 16, max(20000, sum(max(x, 0) for x in new)) + 5, in_place=True)


def test_assign_most_sequences_in_place(cuda_device):
    rng = np.random.default_rng(9)
    B = 8192
    lens = [int(x) for x in rng.integers(0, 70, B)]
    new = [int(x) for x in rng.choice([-1, 0, 1, 3], B)]
    _check_assign(cuda_device, new, lens, *_state(rng, B, 5, 16, lens, 3000), 16, 3 * B, in_place=True)


# ------------------------------------------------------------------ append

def _append_case(rng, lens, new, Hkv, d, bs, spread=2.0):
    """Keys and values of varying size, their slots in blocks in random order, padding tokens
    (slot -1) before, between and behind."""
    width = [-(-(a + b) // bs) for a, b in zip(lens, new)]
    n_blocks = sum(width) + 2
    perm = rng.permutation(n_blocks)
    slots, at = [-1], 0
    for ln, a, w in zip(lens, new, width):
        for t in range(a):
            slots.append(int(perm[at + (ln + t) // bs]) * bs + (ln + t) % bs)
        at += w
        if rng.random() < 0.3:
            slots.append(-1)
    slots.append(-1)
    N = len(slots)
    x = rng.normal(size=(2, N, Hkv, d)) * np.exp(spread * rng.normal(size=(2, N, Hkv, 1)))
    return n_blocks, slots, torch.tensor(x[0]), torch.tensor(x[1])


def _random_cache(rng, n_blocks, Hkv, bs, d, dtype, dev):
    if dtype == E4M3:
        codes = torch.tensor(rng.integers(0, 256, (n_blocks, Hkv, 2, bs, d)), dtype=torch.uint8)
        codes = torch.where((codes & 127) == 127, torch.zeros_like(codes), codes).view(E4M3)
    else:
        codes = torch.tensor(rng.integers(-127, 128, (n_blocks, Hkv, 2, bs, d)), dtype=torch.int8)
    scales = torch.tensor(np.exp2(rng.integers(-9, -3, (n_blocks, Hkv, 2))), dtype=FP32)
    return codes.to(dev), scales.to(dev)


def _check_append(k, v, slots, cache, scales, k_dev=None, v_dev=None):
    dev = cache.device
    values, s64 = ref.decode(cache), scales.cpu().double().numpy()
    ops.kv_cache_append(k.to(dev) if k_dev is None else k_dev, v.to(dev) if v_dev is None else v_dev, i32(slots, dev), cache, scales)
    ref.append(k.double().numpy(), v.double().numpy(), slots, values, s64, cache.dtype)
    np.testing.assert_array_equal(scales.cpu().double().numpy(), s64, err_msg="scales")
    np.testing.assert_array_equal(ref.decode(cache), values, err_msg="codes")


@pytest.mark.parametrize("kv", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_append_mixed_runs(bs, d, dtype, kv, cuda_device):
    """Runs of 1 to several blocks that begin anywhere in a block, for few and for many tokens."""
    rng = np.random.default_rng(bs + d)
    for lens, new, Hkv in (([0, 5, bs - 1, bs, 3 * bs + 7], [1, 1, 2, 1, 3], 2),
                           ([0, 0, 1, bs // 2, bs - 3, 40], [3 * bs, bs + 1, 2 * bs, 5, 4, 2 * bs], 3),
                           ([int(x) for x in rng.integers(0, 2 * bs, 150)], [int(x) for x in rng.integers(0, 60, 150)], 2)):
        n_blocks, slots, k, v = _append_case(rng, lens, new, Hkv, d, bs)
        cache, scales = _random_cache(rng, n_blocks, Hkv, bs, d, kv, cuda_device)
        _check_append(k.to(dtype), v.to(dtype), slots, cache, scales)


@pytest.mark.parametrize("kv", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
def test_append_many_single_tokens(many, kv, cuda_device):
    """Decode steps: each token its own run, some raising their block's scale."""
    rng = np.random.default_rng(5)
    B, Hkv = (1200, 8) if many else (40, 2)
    lens = [int(x) for x in rng.integers(0, 64, B)]
    n_blocks, slots, k, v = _append_case(rng, lens, [1] * B, Hkv, 64, 32, spread=3.0)
    cache, scales = _random_cache(rng, n_blocks, Hkv, 32, 64, kv, cuda_device)
    _check_append(k.to(BF16), v.to(BF16), slots, cache, scales)


@pytest.mark.parametrize("kv", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("n", [2, 20])
def test_append_infinities_nan_zero_and_tiny(n, kv, cuda_device):
    """Infinities and NaN do not move a scale; all-zero and tiny tokens take the smallest one."""
    rng = np.random.default_rng(6)
    Hkv, d, bs = 6, 64, 32
    k, v = torch.tensor(rng.normal(size=(2, n, Hkv, d)))
    k[0, 0, 3], k[1, 0, 5], k[0, 0, 7] = float("inf"), float("-inf"), float("nan")
    k[:, 1] = 0.0
    k[:, 2] *= 2.0 ** -80
    v[:, 3] = float("nan")
    v[:, 4] *= 2.0 ** 100
    v[0, 5, 0] = -448.0 * 2 ** 10
    for off in (0, 3):
        cache, scales = _random_cache(rng, 3, Hkv, bs, d, kv, cuda_device)
        _check_append(k.float(), v.float(), list(range(bs + off, bs + off + n)), cache, scales)


def test_append_leaves_out_slots_outside_the_cache(cuda_device):
    rng = np.random.default_rng(7)
    k, v = (torch.tensor(x).to(BF16) for x in rng.normal(size=(2, 6, 2, 64)))
    cache, scales = _random_cache(rng, 3, 2, 16, 64, INT8, cuda_device)
    _check_append(k, v, [-1, 47, 48, -2147483648, 2147483647, 16], cache, scales)
    before = cache.clone(), scales.clone()
    _check_append(k, v, [-1] * 6, cache, scales)
    assert torch.equal(before[0], cache) and torch.equal(before[1], scales)
    ops.kv_cache_append(k[:0].to(cuda_device), v[:0].to(cuda_device), i32(np.zeros(0), cuda_device), cache, scales)
    assert torch.equal(before[0], cache)


def test_append_strided_tokens(cuda_device):
    """Keys and values as slices of one fused projection."""
    rng = np.random.default_rng(8)
    qkv = torch.tensor(rng.normal(size=(50, 4 + 2 + 2, 128))).to(BF16)
    dev_qkv = qkv.to(cuda_device)
    cache, scales = _random_cache(rng, 5, 2, 32, 128, E4M3, cuda_device)
    _check_append(qkv[:, 4:6], qkv[:, 6:], list(range(70, 120)), cache, scales, dev_qkv[:, 4:6], dev_qkv[:, 6:])


def test_append_under_a_scale_that_is_no_power_of_two(cuda_device):
    """A cache from elsewhere: its larger scale stays and new tokens are divided by it."""
    rng = np.random.default_rng(10)
    dev = cuda_device
    cache, scales = _random_cache(rng, 2, 1, 16, 64, INT8, dev)
    scales[:] = 0.3
    k, v = (torch.tensor(x).float() for x in rng.normal(size=(2, 3, 1, 64)))
    ops.kv_cache_append(k.to(dev), v.to(dev), i32([4, 5, 6], dev), cache, scales)
    assert torch.equal(scales.cpu(), torch.full((2, 1, 2), 0.3))
    want = torch.stack([k[:, 0], v[:, 0]]).div(torch.tensor(0.3)).round().clamp(-127, 127).to(torch.int8)
    assert torch.equal(cache[0, 0, :, 4:7].cpu(), want)


# ------------------------------------------------------------------ attention

def _attention_case(rng, lens, Hkv, bs, d, kv, dev, spread=0.4, stale=True):
    """A cache of normal tokens whose size varies; slots behind a sequence's last token, and blocks
    of no sequence, hold arbitrary bytes (NaN codes among them)."""
    width = max(1, max(-(-n // bs) for n in lens)) + 1
    need = [-(-n // bs) for n in lens]
    n_blocks = sum(need) + 2
    perm = rng.permutation(n_blocks)
    table, at = np.full((len(lens), width), -1), 0
    x = rng.normal(size=(n_blocks, Hkv, 2, bs, d)) * np.exp(spread * rng.normal(size=(n_blocks, Hkv, 2, bs, 1)))
    amax = np.abs(x).max(axis=(3, 4))
    scales = np.exp2(np.ceil(np.log2(amax / ref.QMAX[kv])))
    values = ref.to_code_values(x / scales[..., None, None], kv)
    live = np.zeros((n_blocks, bs), bool)
    for s, k in enumerate(need):
        table[s, :k] = perm[at:at + k]
        for j in range(k):
            live[perm[at + j], :min(bs, lens[s] - j * bs)] = True
        at += k
    codes = torch.tensor(values).float().to(kv).view(torch.uint8)
    if stale:
        junk = torch.tensor(rng.choice([0x7F, 0xFF, 0x80, 3, 200], codes.shape), dtype=torch.uint8)
        codes = torch.where(torch.tensor(live)[:, None, None, :, None], codes, junk)
        values = np.where(live[:, None, None, :, None], values, 0.0)
    return codes.view(kv).to(dev), torch.tensor(scales).float().to(dev), table, values, scales


def _close(out, want, dtype, d, what=""):
    got = out.detach().cpu().double().numpy().reshape(want[0].shape)
    tol = ref.attention_tolerance(want, dtype, d)
    bad = ~(np.abs(got - want[0]) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - want[0]) / tol):.3g} times the "
                           f"tolerance, {np.isnan(got).sum()} NaN")


def _run_attention(rng, dev, lens, nq, G, Hkv, d, bs, kv, dtype, **kw):
    cache, scales, table, values, s64 = _attention_case(rng, lens, Hkv, bs, d, kv, dev, **kw)
    q = torch.tensor(rng.normal(size=(len(lens), nq, Hkv * G, d))).to(dtype)
    out = ops.cached_attention(q.to(dev), cache, scales, i32(table, dev), i32(lens, dev))
    torch.cuda.synchronize()
    assert ops.cached_attention_status() == ops.LIGER_OK
    _close(out, ref.attention(q.double().numpy(), values, s64, table, lens), dtype, d)


RAGGED = [1, 0, 63, 64, 65, 200, 16, 17, 129, 1000]


@pytest.mark.parametrize("kv", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_attention_ragged(bs, d, dtype, kv, cuda_device):
    _run_attention(np.random.default_rng(bs + d), cuda_device, RAGGED, 1, 4, 2, d, bs, kv, dtype)


@pytest.mark.parametrize("nq,G", [(1, 1), (1, 8), (1, 9), (2, 4), (3, 5), (4, 4), (7, 1), (16, 1), (16, 8), (5, 7)])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_attention_new_tokens_and_groups(nq, G, dtype, cuda_device):
    """Query rows from one to many tiles; sequences shorter than the new tokens (rows that see nothing)."""
    _run_attention(np.random.default_rng(nq * G), cuda_device, RAGGED, nq, G, 3, 128, 16, E4M3, dtype)


@pytest.mark.parametrize("lens", [[1], [64], [5000], [30000], [0, 0, 0], [0, 1, 0]], ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_attention_one_sequence_and_empty_ones(lens, d, cuda_device):
    _run_attention(np.random.default_rng(3), cuda_device, lens, 1, 4, 1, d, 64, E4M3, BF16)


def test_attention_many_sequences(cuda_device):
    """More sequences than CTAs, most of them short."""
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(0, 70, 700)]
    _run_attention(rng, cuda_device, lens, 1, 2, 2, 64, 32, INT8, BF16)


def test_attention_most_sequences(cuda_device):
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 20, 8192)]
    _run_attention(rng, cuda_device, lens, 1, 1, 1, 128, 16, INT8, BF16)


def test_attention_most_sequences_of_many_rows(cuda_device):
    """The prefix sums of 8192 sequences beside the largest stages and parts: one CTA an SM."""
    rng = np.random.default_rng(25)
    lens = [int(x) for x in rng.integers(0, 6, 8192)]
    lens[77], lens[8191] = 300, 1000
    _run_attention(rng, cuda_device, lens, 4, 4, 1, 128, 16, E4M3, FP32)


@pytest.mark.parametrize("seed", range(24))
def test_attention_drawn_cases(seed, cuda_device):
    """Sizes drawn over the whole range: units of one tile to many, split and whole, stretches that
    end in a unit, between units and behind the last one."""
    rng = np.random.default_rng(1000 + seed)
    B = int(np.exp(rng.uniform(0, np.log(60))))
    top = int(np.exp(rng.uniform(0, np.log(60000 // B))))
    lens = [int(x) for x in rng.integers(0, top + 1, B)]
    d, G = int(rng.choice([64, 128])), int(rng.choice([1, 2, 3, 4, 5, 8, 17]))
    _run_attention(rng, cuda_device, lens, int(rng.choice([1, 1, 2, 4, 7, 16])), G, int(rng.choice([1, 2, 3])), d,
                   int(rng.choice([16, 32, 64, 128])), E4M3 if rng.random() < 0.5 else INT8, BF16 if rng.random() < 0.6 else FP32)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_attention_peaked_scores_and_unlike_scales(dtype, cuda_device):
    """Scores far apart (the reference is raised again and again, late in the sequence too), and
    value scales that differ by many powers of two between blocks."""
    rng = np.random.default_rng(6)
    dev = cuda_device
    lens, Hkv, d, bs, G = [700, 333], 2, 64, 16, 4
    cache, scales, table, values, s64 = _attention_case(rng, lens, Hkv, bs, d, E4M3, dev, stale=False)
    s64 = s64 * np.exp2(rng.integers(-6, 7, s64.shape) * np.array([0.5, 4.0]).reshape(1, 1, 2) // 1)
    q = torch.tensor(rng.normal(size=(2, 1, Hkv * G, d)) * np.exp2(rng.integers(-12, 5, (2, 1, Hkv * G, 1)))).to(dtype)
    out = ops.cached_attention(q.to(dev), cache, torch.tensor(s64).float().to(dev), i32(table, dev), i32(lens, dev))
    _close(out, ref.attention(q.double().numpy(), values, s64, table, lens), dtype, d)


def test_attention_scales_at_the_ends_of_their_range(cuda_device):
    """Key and value scales from 2^-64 to 2^60 in one sequence: the row's reference and its sum stay finite."""
    rng = np.random.default_rng(16)
    dev, lens, Hkv, d, bs = cuda_device, [80], 1, 64, 16
    cache, _, table, values, s64 = _attention_case(rng, lens, Hkv, bs, d, INT8, dev, stale=False)
    s64[..., 0] = 2.0 ** -8
    s64[..., 1] = np.resize(np.exp2([-64.0, 0.0, 60.0, -20.0, 30.0]), s64.shape[:2])
    q = torch.tensor(rng.normal(size=(1, 1, 2, d))).to(BF16)
    out = ops.cached_attention(q.to(dev), cache, torch.tensor(s64).float().to(dev), i32(table, dev), i32(lens, dev))
    _close(out, ref.attention(q.double().numpy(), values, s64, table, lens), BF16, d)


def test_attention_entries_that_are_no_block(cuda_device):
    """Tokens of such an entry are not there; a sequence of only such entries gets zeros."""
    rng = np.random.default_rng(7)
    dev = cuda_device
    lens = [100, 70, 40]
    cache, scales, table, values, s64 = _attention_case(rng, lens, 2, 16, 64, E4M3, dev)
    table[0, 2], table[0, 6], table[1, 0], table[2, :] = -1, 10 ** 6, -2147483648, values.shape[0]
    q = torch.tensor(rng.normal(size=(3, 2, 4, 64))).to(BF16)
    out = ops.cached_attention(q.to(dev), cache, scales, i32(table, dev), i32(lens, dev))
    want = ref.attention(q.double().numpy(), values, s64, table, lens)
    _close(out, want, BF16, 64)
    assert not out[2].any()


def test_attention_lengths_outside_the_table(cuda_device):
    rng = np.random.default_rng(8)
    dev = cuda_device
    lens = [48, 32]
    cache, scales, table, values, s64 = _attention_case(rng, lens, 1, 16, 64, INT8, dev)
    table = table[:, :3]
    table[1, 2] = table[0, 0]
    q = torch.tensor(rng.normal(size=(2, 1, 2, 64))).to(BF16)
    out = ops.cached_attention(q.to(dev), cache, scales, i32(table, dev), i32([-5, 2 ** 31 - 1], dev))
    assert not out[0].any()
    _close(out[1:], ref.attention(q[1:].double().numpy(), values, s64, table[1:], [48]), BF16, 64)


def test_attention_nan_code_of_a_later_token(cuda_device):
    """A NaN among the newest tokens reaches the queries that see it and no others."""
    rng = np.random.default_rng(9)
    dev = cuda_device
    lens = [77]
    cache, scales, table, values, s64 = _attention_case(rng, lens, 1, 16, 64, E4M3, dev)
    raw = cache.view(torch.uint8)
    blk, off = int(table[0, 75 // 16]), 75 % 16
    raw[blk, 0, :, off] = 0x7F
    q = torch.tensor(rng.normal(size=(1, 4, 3, 64))).to(BF16)
    out = ops.cached_attention(q.to(dev), cache, scales, i32(table, dev), i32(lens, dev))
    assert out[0, 2:].isnan().all()
    want = ref.attention(q[:, :2].double().numpy(), values, s64, table, [75])
    _close(out[:, :2], want, BF16, 64)


def test_attention_strided_queries_and_out(cuda_device):
    rng = np.random.default_rng(10)
    dev = cuda_device
    lens = [40, 300, 7]
    cache, scales, table, values, s64 = _attention_case(rng, lens, 2, 32, 128, E4M3, dev)
    qkv = torch.tensor(rng.normal(size=(3, 12, 128))).to(BF16)
    d = qkv.to(dev)
    out = torch.empty(3, 8, 128, dtype=BF16, device=dev)
    assert ops.cached_attention(d[:, :8], cache, scales, i32(table, dev), i32(lens, dev), out=out) is out
    _close(out, ref.attention(qkv[:, None, :8].double().numpy(), values, s64, table, lens), BF16, 128)
    q4 = torch.tensor(rng.normal(size=(3, 2, 12, 128))).to(BF16)
    out = ops.cached_attention(q4.to(dev)[:, :, 4:], cache, scales, i32(table, dev), i32(lens, dev))
    _close(out, ref.attention(q4[:, :, 4:].double().numpy(), values, s64, table, lens), BF16, 128)


def test_attention_is_the_same_every_time(cuda_device):
    """Splits are joined in a fixed order: repeated calls and a shared dirty workspace change no bit."""
    rng = np.random.default_rng(11)
    dev = cuda_device
    lens = [3000, 1, 777]
    cache, scales, table, _, _ = _attention_case(rng, lens, 2, 16, 128, INT8, dev)
    q = torch.tensor(rng.normal(size=(3, 8, 128))).to(BF16).to(dev)
    ws = torch.full((ops.cached_attention_workspace_size(128),), 0xFF, dtype=torch.uint8, device=dev)
    args = (cache, scales, i32(table, dev), i32(lens, dev))
    first = ops.cached_attention(q, *args)
    for _ in range(5):
        assert torch.equal(first, ops.cached_attention(q, *args, workspace=ws))


def test_attention_offsets_beyond_32_bits(cuda_device):
    """Blocks whose bytes lie beyond 4 GiB of the cache and beyond 2^31 slots' halves."""
    rng = np.random.default_rng(12)
    dev = cuda_device
    n_blocks, Hkv, bs, d = 320000, 1, 64, 128                       # 5.2 GB
    cache = torch.zeros(n_blocks, Hkv, 2, bs, d, dtype=torch.int8, device=dev)
    scales = torch.ones(n_blocks, Hkv, 2, dtype=FP32, device=dev)
    n = 150
    blocks = [n_blocks - 1, 270000, n_blocks - 2]
    slots = [blocks[t // bs] * bs + t % bs for t in range(n)]
    k, v = (torch.tensor(x).to(BF16) for x in rng.normal(size=(2, n, Hkv, d)))
    ops.kv_cache_append(k.to(dev), v.to(dev), i32(slots, dev), cache, scales)
    q = torch.tensor(rng.normal(size=(1, 1, 4, d))).to(BF16)
    out = ops.cached_attention(q.to(dev), cache, scales, i32([blocks], dev), i32([n], dev))
    small, s64 = np.zeros((3, 1, 2, bs, d)), np.ones((3, 1, 2))
    ref.append(k.double().numpy(), v.double().numpy(), list(range(n)), small, s64, INT8)
    np.testing.assert_array_equal(ref.decode(cache[blocks]), small)
    _close(out, ref.attention(q.double().numpy(), small, s64, np.array([[0, 1, 2]]), [n]), BF16, d)


# ------------------------------------------------------------------ together, and as they are called

def _step(c, new, k, v, q, n_slots, bufs=None):
    """One step as a server runs it: the state advances in place."""
    bs = c["cache"].shape[3]
    slots, cu, _, _ = ops.kv_cache_assign(new, c["seq_lens"], c["block_table"], c["free_blocks"], c["free_span"], bs, n_slots,
                                          seq_lens_out=c["seq_lens"], free_span_out=c["free_span"])
    ops.kv_cache_append(k, v, slots, c["cache"], c["scales"])
    return ops.cached_attention(q, c["cache"], c["scales"], c["block_table"], c["seq_lens"])


@pytest.mark.parametrize("kv", [E4M3, INT8], ids=["e4m3", "int8"])
def test_prefill_then_decode_steps(kv, cuda_device):
    """Prompts through the causal attention and into the cache, then decode steps in which one
    sequence ends and a new one takes its blocks.  Every step is held to 64-bit attention over
    the cache's own values, and the cache to the reference's."""
    rng = np.random.default_rng(20)
    dev = cuda_device
    B, Hq, Hkv, d, bs = 3, 8, 2, 64, 16
    c = ops.kv_cache_new(20, Hkv, d, bs, B, 160, dtype=kv, device=dev)
    table, ring, span, lens = c["block_table"].tolist(), c["free_blocks"].tolist(), c["free_span"].tolist(), [0] * B
    values, s64 = np.zeros((20, Hkv, 2, bs, d)), np.ones((20, Hkv, 2))
    prompts = [100, 33, 64]
    plan = [prompts] + [[1, 1, 1]] * 5 + [[1, -1, 1]] + [[1, 70, 1]] + [[1, 1, 1]] * 12
    for i, new in enumerate(plan):
        N = sum(max(x, 0) for x in new)
        k, v = (torch.tensor(x).to(BF16) for x in rng.normal(size=(2, N, Hkv, d)))
        q = torch.tensor(rng.normal(size=(B, Hq, d))).to(BF16)
        if i == 0:      # the prompt's own outputs: causal attention on the unquantised keys
            qp = torch.tensor(rng.normal(size=(1, N, Hq, d))).to(BF16)
            cu = i32(np.cumsum([0] + new), dev)
            assert ops.full_causal_attention(qp.to(dev), k[None].to(dev), v[None].to(dev), cu_seqlens=cu).shape == qp.shape
        out = _step(c, i32(new, dev), k.to(dev), v.to(dev), q.to(dev), N)
        slots, _, lens, span = ref.assign(new, lens, table, ring, span, bs, N)
        ref.append(k.double().numpy(), v.double().numpy(), slots, values, s64, kv)
        assert c["seq_lens"].tolist() == lens and c["free_span"].tolist() == span
        np.testing.assert_array_equal(ref.decode(c["cache"]), values)
        _close(out, ref.attention(q[:, None].double().numpy(), values, s64, np.array(table), lens), BF16, d, f"step {i}")
    # the quantised cache stands for the keys: the step agrees with unquantised attention within the codes' half steps
    assert ops.cached_attention_status() == ops.LIGER_OK


def test_captured_steps_sharing_a_workspace(cuda_device):
    """A decode step captured into a CUDA graph and replayed equals the same steps run eagerly; a
    second graph uses the same workspace in between."""
    rng = np.random.default_rng(21)
    dev = cuda_device
    B, Hq, Hkv, d, bs, steps = 5, 8, 2, 128, 16, 20

    def fresh():
        c = ops.kv_cache_new(40, Hkv, d, bs, B, 64, device=dev)
        k0, v0 = torch.randn(2, 100, Hkv, d, device=dev, generator=torch.Generator(dev).manual_seed(1)).to(BF16)
        slots = ops.kv_cache_assign(i32([20] * B, dev), c["seq_lens"], c["block_table"], c["free_blocks"], c["free_span"], bs,
                                    100, seq_lens_out=c["seq_lens"], free_span_out=c["free_span"])[0]
        ops.kv_cache_append(k0, v0, slots, c["cache"], c["scales"])
        return c

    ks, vs = (torch.tensor(x).to(BF16).to(dev) for x in rng.normal(size=(2, steps, B, Hkv, d)))
    qs = torch.tensor(rng.normal(size=(steps, B, Hq, d))).to(BF16).to(dev)
    new = i32([1] * B, dev)
    c = fresh()
    want = [_step(c, new, ks[i], vs[i], qs[i], B).clone() for i in range(steps)]
    state = [c[x].clone() for x in ("cache", "scales", "block_table", "seq_lens", "free_span")]

    c = fresh()
    k, v, q = (torch.empty_like(x[0]) for x in (ks, vs, qs))
    ws = torch.empty(ops.cached_attention_workspace_size(d), dtype=torch.uint8, device=dev)
    slots, out, out2 = torch.empty(B, dtype=torch.int32, device=dev), torch.empty_like(q), torch.empty_like(q)
    cu = torch.empty(B + 1, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        ops.kv_cache_assign(new, c["seq_lens"], c["block_table"], c["free_blocks"], c["free_span"], bs, B, slot_map=slots,
                            cu_new=cu, seq_lens_out=c["seq_lens"], free_span_out=c["free_span"])
        ops.kv_cache_append(k, v, slots, c["cache"], c["scales"])
        ops.cached_attention(q, c["cache"], c["scales"], c["block_table"], c["seq_lens"], out=out, workspace=ws)
    with torch.cuda.graph(g2):
        ops.cached_attention(q, c["cache"], c["scales"], c["block_table"], c["seq_lens"], out=out2, workspace=ws)
    for i in range(steps):
        k.copy_(ks[i]); v.copy_(vs[i]); q.copy_(qs[i])
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]) and torch.equal(out2, want[i]), i
    for x, w in zip(("cache", "scales", "block_table", "seq_lens", "free_span"), state):
        assert torch.equal(c[x].view(torch.uint8) if x == "cache" else c[x], w.view(torch.uint8) if x == "cache" else w), x


def test_two_streams_at_once(cuda_device):
    """Calls on two streams, each with its own workspace, do not disturb one another."""
    rng = np.random.default_rng(22)
    dev = cuda_device
    cases = []
    for lens in ([2000, 900], [1500, 64, 3]):
        cache, scales, table, _, _ = _attention_case(rng, lens, 2, 32, 128, E4M3, dev)
        q = torch.tensor(rng.normal(size=(len(lens), 8, 128))).to(BF16).to(dev)
        args = (q, cache, scales, i32(table, dev), i32(lens, dev))
        cases.append((args, ops.cached_attention(*args), torch.cuda.Stream(dev)))
    torch.cuda.synchronize()
    outs = [[ops.cached_attention(*args, stream=s) for _ in range(10)] for _ in range(3) for args, _, s in cases]
    torch.cuda.synchronize()
    for i, got in enumerate(outs):
        assert all(torch.equal(x, cases[i % 2][1]) for x in got)


def test_writes_stay_inside_their_tensors(cuda_device):
    rng = np.random.default_rng(23)
    dev = cuda_device
    B, Hq, Hkv, d, bs, n = 4, 12, 3, 64, 16, 9
    lens, new = [15, 0, 31, 16], [2, 5, 1, 1]
    table, ring, span = _state(rng, B, 4, bs, lens, n - 5)
    g = {x: guarded_like(i32(y, dev)) for x, y in dict(new=new, lens=lens, table=table, ring=ring, span=span).items()}
    g["slots"], g["cu"] = Guarded((11,), torch.int32, dev), Guarded((B + 1,), torch.int32, dev)
    ops.kv_cache_assign(g["new"].tensor, g["lens"].tensor, g["table"].tensor, g["ring"].tensor, g["span"].tensor, bs, 11,
                        slot_map=g["slots"].tensor, cu_new=g["cu"].tensor, seq_lens_out=g["lens"].tensor,
                        free_span_out=g["span"].tensor)
    cache, scales = _random_cache(rng, n, Hkv, bs, d, INT8, dev)
    g["cache"], g["scales"] = guarded_like(cache), guarded_like(scales)
    for x in "kv":
        g[x] = guarded_like(torch.tensor(rng.normal(size=(11, Hkv, d))).to(BF16).to(dev))
    ops.kv_cache_append(g["k"].tensor, g["v"].tensor, g["slots"].tensor, g["cache"].tensor, g["scales"].tensor)
    g["q"] = guarded_like(torch.tensor(rng.normal(size=(B, 3, Hq, d))).to(BF16).to(dev))
    g["out"] = Guarded((B, 3, Hq, d), BF16, dev)
    g["ws"] = Guarded((ops.cached_attention_workspace_size(d),), torch.uint8, dev)
    ops.cached_attention(g["q"].tensor, g["cache"].tensor, g["scales"].tensor, g["table"].tensor, g["lens"].tensor,
                         out=g["out"].tensor, workspace=g["ws"].tensor)
    torch.cuda.synchronize()
    for name, x in g.items():
        assert x.intact(), f"{name}: a write beyond the tensor"
    want = ref.attention(g["q"].tensor.cpu().double().numpy(), ref.decode(g["cache"].tensor), g["scales"].tensor.cpu().double().numpy(),
                         np.array(g["table"].tensor.cpu()), g["lens"].tensor.tolist())
    _close(g["out"].tensor, want, BF16, d)


def test_launches_are_counted(cuda_device):
    rng = np.random.default_rng(24)
    cache, scales, table, _, _ = _attention_case(rng, [20], 1, 16, 64, INT8, cuda_device)
    q = torch.zeros(1, 2, 64, dtype=BF16, device=cuda_device)
    before = ops.kernel_launches()
    ops.cached_attention(q, cache, scales, i32(table, cuda_device), i32([20], cuda_device))
    assert ops.kernel_launches() == before + 2


def test_timing_events_bracket_the_kernels(cuda_device):
    """liger_set_timing_events brackets each operator's kernel, as it does the other entry points'."""
    dev = cuda_device
    c = ops.kv_cache_new(8, 2, 64, 16, 3, 32, device=dev)
    k = torch.ones(3, 2, 64, dtype=BF16, device=dev)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record(); b.record()
    new = i32([1, 1, 1], dev)
    calls = [lambda: ops.kv_cache_assign(new, c["seq_lens"], c["block_table"], c["free_blocks"], c["free_span"], 16, 3,
                                         seq_lens_out=c["seq_lens"], free_span_out=c["free_span"]),
             lambda: ops.kv_cache_append(k, k, i32([0, 16, 32], dev), c["cache"], c["scales"]),
             lambda: ops.cached_attention(k, c["cache"], c["scales"], c["block_table"], c["seq_lens"])]
    for call in calls:
        ops.set_timing_events(a, b)
        call()
        ops.set_timing_events(None, None)
        torch.cuda.synchronize()
        assert 0 < a.elapsed_time(b) < 1000


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("order", [[-64, 100], [100, -64], [-64, 0, 100, -30, 60], [100, -64, -64, -64, -64, -64, 20]], ids=str)
@pytest.mark.parametrize("joined", [False, True], ids=["one_cta", "joined"])
def test_attention_value_scales_far_apart(joined, order, dtype, cuda_device):
    """A block of zero values (scale 2^-64) beside one of scale 2^100: its tokens weigh what their scores say, in one
    slice, over slices and tiles, and where the parts of several CTAs are joined."""
    rng = np.random.default_rng(28)
    dev, Hkv, d, bs = cuda_device, 1, 64, 16
    reps = 64 if joined else 1     # (of each block of the order, side by side)
    lens = [len(order) * reps * bs - 5]
    cache, _, table, values, s64 = _attention_case(rng, lens, Hkv, bs, d, INT8, dev, stale=False)
    s64[..., 0] = 2.0 ** -8
    for j, e in enumerate(np.repeat(order, reps)):
        s64[table[0, j], :, 1] = 2.0 ** int(e)
        if e == -64:
            values[table[0, j], :, 1] = 0.0
            cache[int(table[0, j]), :, 1] = 0
    q = torch.tensor(rng.normal(size=(1, 1, 2, d))).to(dtype)
    out = ops.cached_attention(q.to(dev), cache, torch.tensor(s64).float().to(dev), i32(table, dev), i32(lens, dev))
    want = ref.attention(q.double().numpy(), values, s64, table, lens)
    # a weight's exponent is the score less the row's reference, which holds the value scale: up to 2^8 in size here, so
    # that its rounding, half a step of at most 2^-16, moves numerator and sum by 2^-17 each
    got = out.cpu().double().numpy()
    tol = ref.attention_tolerance(want, dtype, d) + 2 * 2.0 ** -17 * want[1]
    assert (np.abs(got - want[0]) <= tol).all(), np.nanmax(np.abs(got - want[0]) / tol)


def test_append_then_attention_of_zero_and_huge_values(cuda_device):
    """The same through the append: fp32 values of 2^100 in one block, zeros in the next, equal scores."""
    dev, d, bs = cuda_device, 64, 16
    c = ops.kv_cache_new(2, 1, d, bs, 1, 2 * bs, device=dev)
    v = torch.zeros(2 * bs, 1, d, device=dev)
    v[:bs] = 2.0 ** 100
    ops.kv_cache_append(torch.ones(2 * bs, 1, d, device=dev), v, i32(range(2 * bs), dev), c["cache"], c["scales"])
    out = ops.cached_attention(torch.ones(1, 1, d, device=dev), c["cache"], c["scales"], i32([[0, 1]], dev), i32([2 * bs], dev))
    # equal scores give equal weights, and 2^100 is a code: the mean, off by the sums' roundings alone
    assert ((out - 2.0 ** 99).abs() <= 2.0 ** 99 * 2.0 ** -20).all()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 5, 5000])
def test_attention_scores_of_huge_magnitude(n, dtype, cuda_device):
    """Scores of -2^110 and beyond are scores: a row's output stays the average of the values that they choose, with
    one token its value."""
    rng = np.random.default_rng(29)
    dev, d, bs = cuda_device, 64, 16
    cache, scales, table, values, s64 = _attention_case(rng, [n], 1, bs, d, INT8, dev)
    cache[:, :, 0] = -4
    scales[..., 0] = 2.0 ** 45
    scales[..., 1] = 2.0 ** -5
    s64[..., 1] = 2.0 ** -5
    q = torch.full((1, 1, d), 2.0 ** 60, dtype=dtype, device=dev)
    out = ops.cached_attention(q, cache, scales, i32(table, dev), i32([n], dev))[0, 0].cpu().double().numpy()
    v = np.concatenate([values[b, 0, 1] * 2.0 ** -5 for b in table[0] if b >= 0])[:n]
    half = torch.finfo(dtype).eps / 2 + 2.0 ** -20   # the output's rounding, the sums'
    assert (out <= v.max(0) + half * np.abs(v).max(0)).all() and (out >= v.min(0) - half * np.abs(v).max(0)).all()
    assert n > 1 or (np.abs(out - v[0]) <= half * np.abs(v[0])).all()
    assert np.abs(out).max() > 0


@pytest.mark.parametrize("n,want", [(16, 3 * 16), (33, -1), (48, 3 * 16)])
def test_assign_next_token_beside_malformed_entries(n, want, cuda_device):
    """A token that starts a block takes it from the ring, whatever stood in the row; one inside a block whose entry is
    no block number has no slot."""
    dev = cuda_device
    slots, _, lens, span = ops.kv_cache_assign(i32([1], dev), i32([n], dev), i32([[5, -1, 99, 3]], dev), i32([3] + [0] * 7, dev),
                                               i32([0, 1], dev), 16, 1)
    assert slots.tolist() == [want] and lens.tolist() == [n + 1]
    assert span.tolist() == ([1, 0] if n % 16 == 0 else [0, 1])


def _half_steps(c, blocks, offs):
    """What the codes of tokens at (blocks, offs) may be off by: half a step under their block's scale, [n, Hkv, 2, d].
    A code that was rounded again when its scale grew is off by half a step of each of its scales, which are powers of two
    below one another: at most twice the last one's for int8.  An e4m3 code keeps its three fraction bits in that, until it
    is subnormal, so its steps add up to no more than those of a value twice as large."""
    scale = c["scales"][blocks].double()[..., None]
    if c["cache"].dtype == INT8:
        return scale.expand(-1, -1, -1, c["cache"].shape[-1])
    code = c["cache"].view(torch.uint8)[blocks, :, :, offs].view(E4M3).double().abs()
    e = torch.clamp(torch.frexp(code)[1] - 1, min=-6)
    return 2 * torch.exp2(e.double() - 4) * scale


@pytest.mark.parametrize("kv", [E4M3, INT8], ids=["e4m3", "int8"])
def test_cached_attention_agrees_with_the_prompt_attention(kv, cuda_device):
    """The newest four tokens of prompts, appended and attended over the cache, against the causal attention over the
    unquantised keys and values, and a token more against 64 bits: within what the codes' half steps can move."""
    rng = np.random.default_rng(31)
    dev, Hq, Hkv, d, bs, lens, nq = cuda_device, 8, 2, 64, 16, [100, 33, 64], 4
    N, B = sum(lens), len(lens)
    q = torch.tensor(rng.normal(size=(1, N, Hq, d)) * 0.25).to(BF16).to(dev)
    k = torch.tensor(rng.normal(size=(1, N, Hkv, d))).to(BF16).to(dev)
    around = rng.choice([-2.0, 2.0], (B, Hkv, d))   # what a sequence's and head's values lie around, far from the others'
    v = torch.tensor(np.repeat(around, lens, 0)[None] + 0.5 * rng.normal(size=(1, N, Hkv, d))).to(BF16).to(dev)
    cu = np.cumsum([0] + lens)
    full = ops.full_causal_attention(q, k, v, cu_seqlens=i32(cu, dev))[0].double()
    c = ops.kv_cache_new(20, Hkv, d, bs, B, 160, dtype=kv, device=dev)
    state = (c["seq_lens"], c["block_table"], c["free_blocks"], c["free_span"])
    put = dict(seq_lens_out=c["seq_lens"], free_span_out=c["free_span"])
    slots = ops.kv_cache_assign(i32(lens, dev), *state, bs, N, **put)[0]
    ops.kv_cache_append(k[0], v[0], slots, c["cache"], c["scales"])
    newest = torch.stack([q[0, cu[s + 1] - nq:cu[s + 1]] for s in range(B)])
    out = ops.cached_attention(newest, c["cache"], c["scales"], c["block_table"], c["seq_lens"]).double()

    def check(got, ks, vs, qs, sl, what, plain=None):
        """got [n, Hq, d], the last n queries qs of a sequence with keys ks, values vs [T, Hkv, d] and slots sl."""
        T, n, G = ks.shape[0], qs.shape[0], Hq // Hkv
        half = _half_steps(c, sl.long() // bs, sl.long() % bs)                          # [T, Hkv, 2, d]
        held = c["cache"].view(torch.uint8)[sl.long() // bs, :, :, sl.long() % bs].view(kv).double() * c["scales"][sl.long() // bs].double()[..., None]
        assert ((held - torch.stack([ks, vs], 2)).abs() <= half).all(), what
        kd, vd, hk, hv = (x.repeat_interleave(G, 1) for x in (ks, vs, half[:, :, 0], half[:, :, 1]))
        mask = torch.arange(T, device=dev) > (T - n + torch.arange(n, device=dev))[:, None]
        x = torch.einsum("nhd,thd->hnt", qs, kd) / d ** 0.5
        w = torch.softmax(x.masked_fill(mask, -np.inf), -1)
        o, spread = torch.einsum("hnt,thd->nhd", w, vd), torch.einsum("hnt,thd->nhd", w, vd.abs())
        # token j's score moves by at most move_j either way, so that its weight grows at most by a factor of e^move_j A and
        # falls at most by its inverse, with A = sum_i w_i e^move_i (their sum falls at most by 1 / A: sum_i w_i e^-move_i is
        # no less, by the means' inequality); then the values move by their half steps
        grown = w * torch.exp(torch.einsum("nhd,thd->hnt", qs.abs(), hk) / d ** 0.5)
        grown = grown * grown.sum(-1, keepdim=True)
        tol = torch.einsum("hnt,thd->nhd", grown - w, vd.abs()) + torch.einsum("hnt,thd->nhd", grown, hv)
        tol = tol + 2.0 ** -7 * (spread + tol)   # weights in bf16 or fp16 and the output's rounding, in either kernel: 2^-8 and less each
        assert ((got - o).abs() <= tol).all(), what
        assert tol.mean() < 0.5 * vd.abs().mean(), "the bound says something"
        if plain is not None:
            assert ((got - plain).abs() <= 2 * tol).all() and ((plain - o).abs() <= tol).all(), what

    kd, vd, qd = k[0].double(), v[0].double(), q[0].double()
    for s in range(B):
        a, b = int(cu[s]), int(cu[s + 1])
        check(out[s], kd[a:b], vd[a:b], qd[b - nq:b], slots[a:b], f"prompt {s}", full[b - nq:b])
    # one more token each
    q1 = torch.tensor(rng.normal(size=(B, Hq, d)) * 0.25).to(BF16).to(dev)
    k1, v1 = (torch.tensor(x).to(BF16).to(dev) for x in (rng.normal(size=around.shape), around + rng.normal(size=around.shape)))
    more = ops.kv_cache_assign(i32([1] * B, dev), *state, bs, B, **put)[0]
    ops.kv_cache_append(k1, v1, more, c["cache"], c["scales"])
    out = ops.cached_attention(q1, c["cache"], c["scales"], c["block_table"], c["seq_lens"]).double()
    for s in range(B):
        a, b = int(cu[s]), int(cu[s + 1])
        check(out[s][None], torch.cat([kd[a:b], k1[s][None].double()]), torch.cat([vd[a:b], v1[s][None].double()]), q1[s][None].double(),
              torch.cat([slots[a:b], more[s:s + 1]]), f"step {s}")


@pytest.mark.parametrize("kv", [E4M3, INT8], ids=["e4m3", "int8"])
def test_drafted_tokens_that_are_turned_down(kv, cuda_device):
    """Steps of up to four drafted tokens a sequence, of which some are kept: the drafts are assigned into new lengths and a
    new span, appended and attended; then the kept ones are assigned again from the old state, which gives the turned down
    ones' blocks back, and appended again.  No block is ever lost or in two rows, and the cache stays the kept tokens'."""
    rng = np.random.default_rng(32)
    dev, B, Hq, Hkv, d, bs, width = cuda_device, 6, 4, 2, 64, 16, 6
    n_blocks = B * width
    c = ops.kv_cache_new(n_blocks, Hkv, d, bs, B, width * bs, dtype=kv, device=dev)
    table, lens, span = c["block_table"], c["seq_lens"], c["free_span"]
    held = [[] for _ in range(B)]   # the kept tokens' keys and values
    for step in range(40):
        new = rng.integers(0, 5, B) if step else rng.integers(1, 40, B)
        if step and step % 7 == 0:
            new[step % B] = -1
        new = np.where(lens.cpu().numpy() + new > width * bs, -1, new)
        count = np.maximum(new, 0)
        kept = np.where(new < 0, -1, rng.integers(0, count + 1)) if step else new
        N = int(count.sum())
        k, v = (torch.tensor(rng.normal(size=(N, Hkv, d))).to(BF16).to(dev) for _ in "kv")
        slots, cu, drafted, _ = ops.kv_cache_assign(i32(new, dev), lens, table, c["free_blocks"], span, bs, N)
        ops.kv_cache_append(k, v, slots, c["cache"], c["scales"])
        q = torch.tensor(rng.normal(size=(B, 4, Hq, d))).to(BF16)
        out = ops.cached_attention(q.to(dev), c["cache"], c["scales"], table, drafted)
        want = ref.attention(q.double().numpy(), ref.decode(c["cache"]), c["scales"].cpu().double().numpy(), table.cpu().numpy(), drafted.tolist())
        _close(out, want, BF16, d, f"drafts of step {step}")
        # the kept ones, from the same lengths and span as before
        at = np.concatenate([cu[s].item() + np.arange(max(kept[s], 0)) for s in range(B)]).astype(int)
        slots, _, lens, span = ops.kv_cache_assign(i32(kept, dev), lens, table, c["free_blocks"], span, bs, len(at))
        ops.kv_cache_append(k[at], v[at], slots, c["cache"], c["scales"])
        assert (slots >= 0).all()
        for s in range(B):
            held[s] = [] if kept[s] < 0 else held[s] + [torch.stack([k[cu[s] + i], v[cu[s] + i]], 1).double() for i in range(kept[s])]
        assert lens.tolist() == [len(x) for x in held]
        used = [int(table[s, j]) for s in range(B) for j in range(-(-len(held[s]) // bs))]
        head, free = span.tolist()
        assert sorted(used + [int(c["free_blocks"][(head + i) % n_blocks]) for i in range(free)]) == list(range(n_blocks)), step
        for s in range(B):
            if held[s]:
                pos = torch.arange(len(held[s]), device=dev)
                blk, off = table[s, pos // bs].long(), pos % bs
                got = c["cache"].view(torch.uint8)[blk, :, :, off].view(kv).double() * c["scales"][blk].double()[..., None]
                assert ((got - torch.stack(held[s])).abs() <= _half_steps(c, blk, off)).all(), step


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_nonfinite_queries_stay_in_their_rows(d, dtype, cuda_device):
    """A NaN or an infinity in one query row reaches no other row of its unit, not even of its own token or head."""
    rng = np.random.default_rng(33)
    dev, lens, nq, G, bs = cuda_device, [40, 3000, 2], 4, 4, 16
    cache, scales, table, values, s64 = _attention_case(rng, lens, 1, bs, d, E4M3, dev)
    q = torch.tensor(rng.normal(size=(3, nq, G, d))).to(dtype)
    want = ref.attention(q.double().numpy(), values, s64, table, lens)
    bad = np.zeros((3, nq, G), bool)
    for s, i, h, x in ((0, 1, 2, "nan"), (1, 0, 0, "inf"), (1, 3, 3, "nan"), (2, 3, 1, "-inf")):
        q[s, i, h, 5] = float(x)
        bad[s, i, h] = True
    out = ops.cached_attention(q.to(dev), cache, scales, i32(table, dev), i32(lens, dev))
    keep = np.where(bad[..., None], 0.0, 1.0)
    got = torch.where(torch.tensor(bad, device=dev)[..., None], torch.zeros_like(out), out)
    _close(got, tuple(w * (keep if w.ndim == 4 else keep[..., 0]) for w in want), dtype, d)
    assert out[0, 1, 2].isnan().all() and out[1, 3, 3].isnan().all()


@pytest.mark.parametrize("nq,Hq,Hkv,d,dtype", [(16, 4096, 1, 64, BF16), (3, 1000, 1, 128, FP32), (1, 4096, 4096, 64, BF16)])
def test_attention_most_rows_and_heads(nq, Hq, Hkv, d, dtype, cuda_device):
    """The largest numbers of rows a kv head, and thousands of kv heads: sampled rows against 64 bits."""
    rng = np.random.default_rng(34)
    dev, lens, bs = cuda_device, [37, 0, 90], 16
    cache, scales, table, values, s64 = _attention_case(rng, lens, Hkv, bs, d, INT8, dev)
    q = torch.tensor(rng.normal(size=(3, nq, Hq, d))).to(dtype)
    out = ops.cached_attention(q.to(dev), cache, scales, i32(table, dev), i32(lens, dev))
    assert not out[1].any()
    for h in [0, Hq - 1] + [int(x) for x in rng.integers(0, Hq, 6)]:
        g = h // (Hq // Hkv)
        _close(out[:, :, h:h + 1], ref.attention(q[:, :, h:h + 1].double().numpy(), values[:, g:g + 1], s64[:, g:g + 1], table, lens), dtype, d)
