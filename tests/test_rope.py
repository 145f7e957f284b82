"""Rotary positions fused with the paged KV write, against the definition in 64
bits; its refusals; the frequency tables of the context scalings."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_211_gb300 as pkv
from paged_kv_cache_211_gb300 import build as pkv_build
from rope_reference import bound, rotate

bf, f16 = torch.bfloat16, torch.float16
HALF_STEP = {bf: 2.0 ** -134, f16: 2.0 ** -25}  # half the smallest subnormal step


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


# ------------------------------------------------------------------ frequencies (host)
def test_plain_linear_and_ntk_frequencies():
    R, j = 64, np.arange(32)
    f, m = pkv.paged_kv_rope_frequencies(R, 10000.0)
    np.testing.assert_array_equal(f.numpy(), (10000.0 ** (-2.0 * j / R)).astype(np.float32))
    assert m == 1.0 and f[0] == 1.0
    f, m = pkv.paged_kv_rope_frequencies(R, 10000.0, "linear", 4.0)
    np.testing.assert_array_equal(f.numpy(), (10000.0 ** (-2.0 * j / R) / 4.0).astype(np.float32))
    f, m = pkv.paged_kv_rope_frequencies(R, 10000.0, "ntk", 8.0)
    # the slowest pair turns `factor` times slower, the fastest as before
    assert f[0] == 1.0 and m == 1.0
    assert f[-1].item() == pytest.approx(10000.0 ** (-62 / 64) / 8.0, rel=1e-6)


def test_yarn_frequencies_keep_fast_pairs_and_divide_slow_ones():
    R, factor, orig = 128, 16.0, 4096
    plain, _ = pkv.paged_kv_rope_frequencies(R)
    f, m = pkv.paged_kv_rope_frequencies(R, scaling="yarn", factor=factor, original_max_position=orig)
    assert m == pytest.approx(0.1 * math.log(factor) + 1.0, rel=1e-6)
    turns = orig * plain.double() / (2 * math.pi)
    ratio = f.double() / plain.double()
    # pairs a whole index inside the ramp's ends (the ends are rounded outwards)
    assert torch.allclose(ratio[turns > 32 * 1.5], torch.ones(1, dtype=torch.float64), rtol=2e-7)
    assert torch.allclose(ratio[turns < 1 / 1.5], torch.full((1,), 1 / factor, dtype=torch.float64),
                          rtol=2e-7)
    assert (ratio[1:] <= ratio[:-1] + 1e-7).all() and (ratio > 1 / factor - 1e-7).all()


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=64, base=1.0),
    dict(rotary_dim=64, base=float("inf")), dict(rotary_dim=64, scaling="linear", factor=0.5),
    dict(rotary_dim=64, scaling="ntk", factor=float("nan")),
    dict(rotary_dim=64, scaling="yarn", factor=2.0),
    dict(rotary_dim=64, scaling="yarn", factor=2.0, original_max_position=4096, beta_fast=1.0,
         beta_slow=2.0),
])
def test_frequencies_refuse(kw):
    with pytest.raises(pkv.PagedKVError) as e:
        pkv.paged_kv_rope_frequencies(**kw)
    assert e.value.status == pkv.PKV_ERR_INVALID_ARG


def test_frequencies_refuse_an_unknown_scaling():
    with pytest.raises(ValueError, match="scaling"):
        pkv.paged_kv_rope_frequencies(64, scaling="log")


# ------------------------------------------------------------------ refusals (no GPU)
def _cpu_args(**over):
    T, Hq, Hkv, D, NB = 3, 4, 2, 64, 5
    a = dict(q=torch.zeros(T, Hq, D, dtype=bf), k_new=torch.zeros(T, Hkv, D, dtype=bf),
             v_new=torch.zeros(T, Hkv, D, dtype=bf), k_cache=torch.zeros(NB, 16, Hkv, D, dtype=bf),
             v_cache=torch.zeros(NB, 16, Hkv, D, dtype=bf),
             positions=torch.zeros(T, dtype=torch.int32),
             slot_mapping=torch.zeros(T, dtype=torch.int64), inv_freq=torch.ones(32),
             q_out=torch.zeros(T, Hq, D, dtype=bf))
    a.update(over)
    return a


@pytest.mark.parametrize("over,msg", [
    (dict(positions=torch.zeros(3, dtype=torch.int64)), "positions must be int32"),
    (dict(positions=torch.zeros(2, dtype=torch.int32)), "positions must be int32"),
    (dict(slot_mapping=torch.zeros(3, dtype=torch.int32)), "slot_mapping must be int64"),
    (dict(inv_freq=torch.ones(33)), "inv_freq must be float32"),
    (dict(inv_freq=torch.ones(32, dtype=torch.float64)), "inv_freq must be float32"),
    (dict(q_out=torch.zeros(3, 4, 64, dtype=f16)), "share one dtype"),
    (dict(q_out=torch.zeros(3, 5, 64, dtype=bf)), "share one dtype"),
    (dict(k_new=torch.zeros(3, 3, 64, dtype=bf)), "k_new/v_new must be shaped"),
    (dict(v_cache=torch.zeros(5, 16, 2, 32, dtype=bf)), "pool shape"),
    (dict(), "must be a CUDA tensor"),
])
def test_rope_write_refuses(over, msg):
    with pytest.raises(ValueError, match=msg):
        pkv.paged_kv_rope_write(**_cpu_args(**over))


def _c_call(**over):
    """The C entry with made-up pointers: every refusal precedes any CUDA call."""
    a = dict(q=1 << 20, k_new=2 << 20, v_new=3 << 20, q_stride=256, k_stride=128, v_stride=128,
             positions=4 << 20, slot_mapping=5 << 20, inv_freq=6 << 20, rope_scale=1.0,
             num_tokens=4, num_q_heads=4, num_kv_heads=2, head_dim=64, rotary_dim=64, layout=0,
             num_blocks=8, q_out=7 << 20, k_cache=8 << 20, v_cache=9 << 20, dtype=1, stream=None)
    a.update(over)
    return pkv.lib().paged_kv_rope_write(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(rotary_dim=63), 1), (dict(rotary_dim=66), 1), (dict(rotary_dim=0), 1),
    (dict(layout=2), 1), (dict(dtype=2), 1), (dict(num_tokens=-1), 1), (dict(num_blocks=0), 1),
    (dict(rope_scale=float("inf")), 1), (dict(rope_scale=float("nan")), 1),
    (dict(q_stride=255), 1), (dict(q_stride=252), 1), (dict(k_stride=132), 1),
    (dict(q=None), 1), (dict(positions=None), 1), (dict(slot_mapping=None), 1),
    (dict(q=(1 << 20) + 8), 1), (dict(q_out=(7 << 20) + 2), 1),
    (dict(head_dim=60, rotary_dim=60, q_stride=240, k_stride=120, v_stride=120), 2),
    (dict(head_dim=520, rotary_dim=64, q_stride=2080, k_stride=1040, v_stride=1040), 2),
    (dict(q_out=(1 << 20) + 512), 1),               # overlaps q, one token on
    (dict(q_out=1 << 20, q_stride=512), 1),         # in place needs contiguous rows
    (dict(q_out=2 << 20), 1), (dict(q_out=(3 << 20) - 1024), 1),   # overlaps k_new / v_new
    (dict(num_tokens=0), 0), (dict(num_tokens=0, positions=None, q=None), 0),
])
def test_rope_write_c_statuses(over, status):
    assert _c_call(**over) == status


# ------------------------------------------------------------------ parity (GPU)
def _case(dev, T, Hq, Hkv, D, dtype, seed, packed=False):
    g = torch.Generator(device=dev).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=dev).to(dtype)
    if packed:
        rows = n(T, (Hq + 2 * Hkv) * D + 8)      # the projection's rows, wider still
        q = rows[:, :Hq * D].view(T, Hq, D)
        k = rows[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        v = rows[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(T, Hkv, D)
    else:
        q, k, v = n(T, Hq, D), n(T, Hkv, D), n(T, Hkv, D)
    NB = T // 16 + 3
    kc, vc = n(NB, 16, Hkv, D), n(NB, 16, Hkv, D)
    return q, k, v, kc, vc


def _check(got, want, size, m, dtype, positions):
    tol = bound(want, size, m, torch.finfo(dtype).eps, HALF_STEP[dtype], positions)
    err = np.abs(got - want)
    assert (err <= tol).all(), f"{(err / tol).max():.3f} of the bound at {np.argmax(err / tol)}"


def _f64(t):
    return t.double().cpu().numpy()


def _run_and_check(dev, T, Hq, Hkv, D, R, dtype, interleaved, packed, pos, seed=0, m=1.0, pad=0,
                   in_place=False, stream=None):
    q, k, v, kc, vc = _case(dev, T, Hq, Hkv, D, dtype, seed, packed)
    freq, _ = pkv.paged_kv_rope_frequencies(R)
    rng = np.random.default_rng(seed)
    slots = rng.permutation(kc.shape[0] * 16)[:T].astype(np.int64)
    if pad:
        slots[::pad] = -1
    live = slots >= 0
    q64, k64, kc0, vc0 = _f64(q), _f64(k), kc.clone(), vc.clone()
    q_out = q if in_place else torch.full((T, Hq, D), 7.0, dtype=dtype, device=dev)
    q_out0 = _f64(q_out)
    pos = np.asarray(pos, np.int64)
    args = (q, k, v, kc, vc, torch.tensor(pos, dtype=torch.int32, device=dev),
            torch.tensor(slots, device=dev), freq.to(dev), q_out)
    torch.cuda.synchronize()
    pkv.paged_kv_rope_write(*args, interleaved=interleaved, rope_scale=m, stream=stream)
    torch.cuda.synchronize()
    assert pkv.pkv_device_status() == 0
    f = freq.numpy()
    want, size = rotate(q64, pos, f, m, interleaved)
    _check(_f64(q_out)[live], want[live], size[live], m, dtype, pos[live])
    np.testing.assert_array_equal(_f64(q_out)[~live], q_out0[~live])
    want, size = rotate(k64, pos, f, m, interleaved)
    rows = kc.view(-1, Hkv, D)
    at = torch.tensor(slots[live], device=dev)
    _check(_f64(rows[at]), want[live], size[live], m, dtype, pos[live])
    # elements behind the rotated part, v, and every other slot: bit for bit
    lv = torch.tensor(np.flatnonzero(live), device=dev)
    ints = lambda t: t.contiguous().view(torch.int16)
    assert torch.equal(ints(rows[at][..., R:]), ints(k[lv][..., R:]))
    assert torch.equal(ints(vc.view(-1, Hkv, D)[at]), ints(v[lv]))
    kc0.view(-1, Hkv, D)[at] = rows[at]
    vc0.view(-1, Hkv, D)[at] = v[lv]
    assert torch.equal(ints(kc), ints(kc0)) and torch.equal(ints(vc), ints(vc0))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [f16, bf])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,R", [
    (1, 1, 1, 64, 64), (1, 16, 8, 128, 128), (5, 32, 8, 128, 64), (37, 7, 7, 64, 32),
    (130, 12, 4, 64, 48), (33, 3, 1, 80, 80), (9, 5, 5, 96, 20), (17, 4, 2, 64, 10),
    (6, 2, 1, 128, 2), (4, 2, 2, 8, 6), (3, 4, 4, 512, 510), (2, 300, 1, 256, 256),
    (2, 1, 1, 512, 2), (300, 40, 8, 128, 128),
])
def test_rope_write_matches_the_definition(cuda_device, T, Hq, Hkv, D, R, dtype, interleaved):
    pos = np.random.default_rng(T).integers(0, 40000, T)
    _run_and_check(cuda_device, T, Hq, Hkv, D, R, dtype, interleaved, packed=T % 2 == 1, pos=pos,
                   seed=T * 7 + D, m=1.0 + 0.25 * interleaved, pad=5 if T > 30 else 0)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_write_far_and_negative_positions(cuda_device, interleaved):
    pos = [0, 1, 65535, 65536, 65537, 1000003, 2 ** 24 - 1, 2 ** 24 + 1, 123456789, 2 ** 31 - 1,
           -1, -65536, -70001]
    _run_and_check(cuda_device, len(pos), 4, 2, 128, 128, f16, interleaved, False, pos, m=0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("R,interleaved", [(128, False), (128, True), (20, False), (2, False)])
def test_rope_write_in_place(cuda_device, R, interleaved):
    _run_and_check(cuda_device, 50, 6, 2, 128, R, bf, interleaved, False, np.arange(50) * 37,
                   in_place=True, pad=7)


@pytest.mark.gpu
def test_rope_write_on_another_stream(cuda_device):
    st = torch.cuda.Stream()
    _run_and_check(cuda_device, 64, 8, 2, 64, 64, bf, False, True, np.arange(64), stream=st)


@pytest.mark.gpu
def test_rope_write_flags_a_slot_past_the_pool(cuda_device):
    dev = cuda_device
    q, k, v, kc, vc = _case(dev, 3, 4, 2, 64, bf, 1)
    before = kc.clone(), vc.clone()
    out = torch.zeros_like(q)
    freq = pkv.paged_kv_rope_frequencies(64, device=dev)[0]
    slots = torch.tensor([kc.shape[0] * 16, -1, 1 << 40], device=dev)
    pkv.paged_kv_rope_write(q, k, v, kc, vc, torch.zeros(3, dtype=torch.int32, device=dev), slots,
                            freq, out)
    assert pkv.pkv_device_status() == pkv.DEV_BAD_SLOT
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1]) and not out.any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [f16, bf])
def test_rope_step_places_each_token(cuda_device, dtype):
    """The single-token form: slots and positions from tables and lengths, empty and
    bad sequences left alone; captured and replayed with other lengths."""
    dev = cuda_device
    B, Hq, Hkv, D, R, NB, MB = 9, 8, 2, 64, 32, 40, 4
    q, k, v, _, _ = _case(dev, B, Hq, Hkv, D, dtype, 3)
    rng = np.random.default_rng(5)
    table = rng.permutation(NB)[:B * MB].reshape(B, MB).astype(np.int32)
    table[7, 1] = NB          # bad id, reached by sequence 7
    table[8, 0] = -1
    freq, _ = pkv.paged_kv_rope_frequencies(R)
    bt = torch.tensor(table, device=dev)
    cl = torch.zeros(B, dtype=torch.int32, device=dev)
    out = torch.zeros(B, Hq, D, dtype=dtype, device=dev)
    slots = torch.zeros(B, dtype=torch.int64, device=dev)
    kc = torch.zeros(NB, 16, Hkv, D, dtype=dtype, device=dev)
    vc = torch.zeros_like(kc)
    fr = freq.to(dev)
    call = lambda: pkv.paged_kv_rope_write_new_tokens(q, k, v, kc, vc, bt, cl, fr, out,
                                                      interleaved=True, slot_mapping_out=slots)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([1, 16, 17, 64, 0, 33, 65, 20, 5], [2, 1, 64, 49, 50, 0, -1, 16, 17]):
        for t in (kc, vc, out):
            t.zero_()
        cl.copy_(torch.tensor(lens, dtype=torch.int32))
        pkv.pkv_device_status()
        graph.replay()
        torch.cuda.synchronize()
        want_slots = []
        for s, n in enumerate(lens):
            b = table[s, (n - 1) // 16] if 0 < n <= MB * 16 else -1
            want_slots.append(int(b) * 16 + (n - 1) % 16 if 0 <= b < NB else -1)
        assert slots.tolist() == want_slots
        flags = pkv.DEV_BAD_LENGTH
        if lens[7] > 16 or 0 < lens[8] <= 16:
            flags |= pkv.DEV_BAD_BLOCK_ID
        assert pkv.pkv_device_status() == flags
        pos = np.maximum(np.array(lens) - 1, 0)
        live = [s for s in range(B) if want_slots[s] >= 0]
        dead = [s for s in range(B) if want_slots[s] < 0]
        wq, sq = rotate(_f64(q), pos, freq.numpy(), 1.0, True)
        _check(_f64(out)[live], wq[live], sq[live], 1.0, dtype, pos[live])
        assert not out[dead].any()
        wk, sk = rotate(_f64(k), pos, freq.numpy(), 1.0, True)
        at = torch.tensor([want_slots[s] for s in live], device=dev)
        _check(_f64(kc.view(-1, Hkv, D)[at]), wk[live], sk[live], 1.0, dtype, pos[live])
        assert torch.equal(vc.view(-1, Hkv, D)[at], v[live])
        assert int((kc.view(-1, Hkv * D) != 0).any(1).sum()) == len(live)
        assert int((vc.view(-1, Hkv * D) != 0).any(1).sum()) == len(live)


@pytest.mark.gpu
def test_rope_write_passes_special_values(cuda_device):
    """Infinities and NaN outside the rotated part and in v are copied bit for bit,
    and one head's NaN stays in its own pair."""
    dev = cuda_device
    q, k, v, kc, vc = _case(dev, 2, 2, 1, 64, bf, 9)
    q[0, 0, 40] = float("nan")
    k[0, 0, 50] = float("-inf")
    v[1, 0, 3] = float("inf")
    q[1, 1, 5] = float("nan")
    out = torch.zeros_like(q)
    freq = pkv.paged_kv_rope_frequencies(32, device=dev)[0]
    slots = torch.tensor([3, 17], device=dev)
    pkv.paged_kv_rope_write(q, k, v, kc, vc, torch.tensor([7, 8], dtype=torch.int32, device=dev),
                            slots, freq, out)
    assert out[0, 0, 40].isnan() and kc[0, 3, 0, 50] == float("-inf")
    assert vc[1, 1, 0, 3] == float("inf")
    nan = out.isnan().nonzero().tolist()
    assert nan == [[0, 0, 40], [1, 1, 5], [1, 1, 21]]
