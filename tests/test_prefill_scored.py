"""Chunked attention with capped and biased scores, windows, prefixes and
documents, against the definition in 64 bits; its refusals."""
import pytest
import torch

import paged_kv_cache_211_gb300 as pkv
from paged_kv_cache_211_gb300 import build as pkv_build
from scored_reference import assert_close, attention

BS = 16
bf, f16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


# ------------------------------------------------------------------ refusals (no GPU)
def _cpu_args(**over):
    B, R, Hq, Hkv, D, NB = 2, 5, 8, 2, 64, 10
    a = dict(q=torch.zeros(R, Hq, D, dtype=bf), k_cache=torch.zeros(NB, 16, Hkv, D, dtype=bf),
             v_cache=torch.zeros(NB, 16, Hkv, D, dtype=bf),
             block_tables=torch.zeros(B, 4, dtype=torch.int32),
             context_lens=torch.ones(B, dtype=torch.int32),
             cu_q_lens=torch.zeros(B + 1, dtype=torch.int32), max_q_len=4, scale=0.125,
             out=torch.zeros(R, Hq, D, dtype=bf), workspace=torch.zeros(1024, dtype=torch.uint8))
    a.update(over)
    return a


@pytest.mark.parametrize("over,msg", [
    (dict(alibi_slopes=torch.zeros(8, dtype=f16)), "alibi_slopes must be float32"),
    (dict(key_starts=torch.zeros(3, dtype=torch.int32)), "key_starts must be int32"),
    (dict(prefix_lens=torch.zeros(2, dtype=torch.int64)), "prefix_lens must be int32"),
    (dict(cu_q_lens=torch.zeros(2, dtype=torch.int32)), "cu_q_lens must be int32"),
    (dict(out=torch.zeros(5, 8, 64, dtype=f16)), "share one dtype"),
    (dict(v_cache=torch.zeros(10, 16, 2, 32, dtype=bf)), "pool shape"),
    (dict(), "must be a CUDA tensor"),  # (the refusal that every well-formed call here meets)
])
def test_prefill_scored_refuses(over, msg):
    with pytest.raises(ValueError, match=msg):
        pkv.paged_attention_prefill_scored(**_cpu_args(**over))


def _c_call(**over):
    a = dict(q=1 << 20, k_cache=2 << 20, v_cache=3 << 20, block_tables=4 << 20,
             max_blocks_per_seq=4, context_lens=5 << 20, cu_q_lens=6 << 20, num_seqs=2,
             max_q_len=8, num_q_rows=12, num_q_heads=8, num_kv_heads=2, head_dim=64, num_blocks=8,
             scale=0.1, softcap=0.0, alibi_slopes=None, window=0, key_starts=None,
             prefix_lens=None, out=7 << 20, workspace=8 << 20, workspace_bytes=1 << 30, dtype=1,
             stream=None)
    a.update(over)
    return pkv.lib().paged_attention_prefill_scored(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(scale=float("nan")), 1), (dict(softcap=-0.5), 1), (dict(softcap=float("inf")), 1),
    (dict(window=-2), 1), (dict(num_q_heads=9), 1), (dict(dtype=2), 1), (dict(num_q_rows=-1), 1),
    (dict(q=None), 1), (dict(cu_q_lens=None), 1), (dict(out=(7 << 20) + 8), 1),
    (dict(num_q_heads=34), 2), (dict(head_dim=80), 2), (dict(max_q_len=1 << 27), 2),
    (dict(max_blocks_per_seq=1 << 27), 2), (dict(num_blocks=1 << 27), 2),
    (dict(workspace=None), 6), (dict(workspace_bytes=100), 6), (dict(workspace=(8 << 20) + 128), 6),
    (dict(num_seqs=0), 0), (dict(max_q_len=0, q=None), 0), (dict(num_q_rows=0, workspace=None), 0),
    (dict(out=1 << 20), 1), (dict(out=(1 << 20) + 12272), 1), (dict(out=(1 << 20) - 12272), 1),
])
def test_prefill_scored_c_statuses(over, status):
    assert _c_call(**over) == status


def test_workspace_size():
    f = pkv.paged_attention_prefill_scored_workspace_bytes
    assert f(0, 8, 8, 2, 64) == 0 and f(1, 8, 8, 2, 96) == 0 and f(1, 8, 8, 3, 64) == 0
    assert f(64, 2048, 32, 8, 128) == 256            # enough items: nothing is split
    assert 1 << 20 < f(1, 4, 8, 1, 128) < 32 << 20


# ------------------------------------------------------------------ parity (GPU)
def make(dev, chunks, lens, Hq, Hkv, D, dtype, seed=0, q_std=1.5, starts=None, window=0,
         prefixes=None, pad_rows=0):
    """As for decode: what no row sees is NaN, table entries of such blocks are -1."""
    g = torch.Generator(device=dev).manual_seed(seed)
    need = [(max(n, 0) + BS - 1) // BS for n in lens]
    MB = max(max(need), 1)
    NB = sum(need) + 5
    perm = torch.randperm(NB, generator=g, device=dev).tolist()
    kc = torch.full((NB * BS, Hkv, D), float("nan"), dtype=dtype, device=dev)
    vc = torch.full((NB * BS, Hkv, D), float("nan"), dtype=dtype, device=dev)
    tables, at = [], 0
    for s, n in enumerate(lens):
        ids = perm[at:at + need[s]]
        at += need[s]
        lo = max(starts[s] if starts is not None else 0, 0,
                 n - chunks[s] - window + 1 if window else 0)
        if chunks[s] > 0 and lo < n:
            t = torch.arange(lo, n, device=dev)
            slots = torch.tensor(ids, device=dev)[t // BS] * BS + t % BS
            kc[slots] = torch.randn(n - lo, Hkv, D, generator=g, device=dev).to(dtype)
            vc[slots] = torch.randn(n - lo, Hkv, D, generator=g, device=dev).to(dtype)
            ids = [-1] * (lo // BS) + ids[lo // BS:]
        else:
            ids = [-1] * len(ids)
        tables.append(ids + [-1] * (MB - need[s]))
    rows = sum(chunks) + pad_rows
    q = (torch.randn(rows, Hq, D, generator=g, device=dev) * q_std).to(dtype)
    return dict(q=q, k_cache=kc.view(NB, BS, Hkv, D), v_cache=vc.view(NB, BS, Hkv, D),
                tables=tables, lens=list(lens), chunks=list(chunks), starts=starts, window=window,
                prefixes=prefixes)


def run(inp, scale, softcap=0.0, slopes=None, stream=None, flags=0, max_chunk=None, cu=None):
    dev = inp["q"].device
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=dev)
    R, Hq, D = inp["q"].shape
    Hkv = inp["k_cache"].shape[2]
    if cu is None:
        cu = [0]
        for c in inp["chunks"]:
            cu.append(cu[-1] + c)
    mx = max_chunk or max(inp["chunks"])
    out = torch.full_like(inp["q"], 3.0)
    ws = pkv.new_prefill_scored_workspace(len(inp["lens"]), mx, Hq, Hkv, D, dev).fill_(255)
    t = [i32(x) for x in (inp["tables"], inp["lens"], cu, inp["starts"], inp["prefixes"])]
    torch.cuda.synchronize()
    pkv.paged_attention_prefill_scored(
        inp["q"], inp["k_cache"], inp["v_cache"], t[0], t[1], t[2], mx, scale, out, ws,
        softcap=softcap, alibi_slopes=slopes, window=inp["window"], key_starts=t[3],
        prefix_lens=t[4], stream=stream)
    torch.cuda.synchronize()
    assert pkv.pkv_device_status() == flags
    return out


def check(inp, scale, softcap=0.0, slopes=None, **kw):
    out = run(inp, scale, softcap, slopes, **kw)
    want, tol = attention(inp["q"], inp["k_cache"], inp["v_cache"], inp["tables"], inp["lens"],
                          inp["chunks"], scale, softcap, slopes, inp["window"], inp["starts"],
                          inp["prefixes"])
    rows = sum(inp["chunks"])
    assert (out[rows:] == 3.0).all()                 # rows behind the last chunk stay
    return assert_close(out[:rows], want[:rows], tol[:rows])


def slopes_of(Hq, dev):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / Hq) for i in range(Hq)], device=dev)


HEADS = [(1, 1, 64), (8, 8, 128), (16, 8, 128), (12, 4, 64), (16, 1, 128), (7, 1, 64), (9, 3, 128),
         (10, 2, 64), (11, 1, 128), (32, 4, 64)]
CHUNKS = [1, 2, 17, 64, 127, 128, 129, 300, 0, 5]
LENS = [1, 100, 17, 90, 127, 1000, 400, 555, 40, 2100]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [f16, bf])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_head_layouts_with_cap_and_bias(cuda_device, Hq, Hkv, D, dtype):
    inp = make(cuda_device, CHUNKS, LENS, Hq, Hkv, D, dtype, seed=Hq + D, pad_rows=3)
    check(inp, D ** -0.5, softcap=20.0, slopes=slopes_of(Hq, cuda_device))


@pytest.mark.gpu
@pytest.mark.parametrize("cap,bias", [(0.0, False), (0.0, True), (30.0, False), (3.0, False),
                                      (3.0, True)])
@pytest.mark.parametrize("D,dtype", [(64, bf), (128, f16)])
def test_cap_and_bias(cuda_device, cap, bias, D, dtype):
    inp = make(cuda_device, CHUNKS, LENS, 8, 4, D, dtype, seed=3, q_std=3.0)
    check(inp, D ** -0.5, softcap=cap, slopes=slopes_of(8, cuda_device) if bias else None)


@pytest.mark.gpu
@pytest.mark.parametrize("chunks,lens", [([4], [5000]), ([1], [1]), ([3, 2], [900, 130]),
                                         ([9] * 7, [2000, 9, 128, 300, 1999, 64, 700])])
@pytest.mark.parametrize("D", [64, 128])
def test_few_rows_over_long_keys_are_split_and_joined(cuda_device, chunks, lens, D):
    inp = make(cuda_device, chunks, lens, 8, 2, D, bf, seed=sum(lens), pad_rows=1)
    check(inp, 0.1, softcap=15.0, slopes=slopes_of(8, cuda_device))
    inp = make(cuda_device, chunks, lens, 6, 2, D, f16, seed=2, window=70,
               starts=[n // 2 for n in lens])
    check(inp, 0.1)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [1, 2, 16, 100, 128, 129, 500, 2 ** 31 - 1])
def test_windows(cuda_device, window):
    inp = make(cuda_device, CHUNKS, LENS, 4, 2, 128, bf, seed=window % 997, window=window)
    check(inp, 0.1, softcap=10.0)
    inp = make(cuda_device, CHUNKS * 8, LENS * 8, 4, 4, 64, f16, seed=5, window=window)
    check(inp, 0.1, slopes=slopes_of(4, cuda_device))


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("reps", [1, 8])
def test_key_starts_and_empty_rows(cuda_device, window, reps):
    starts = [0, -5, 16, 45, 200, 995, 399, 300, 7, 2 ** 31 - 1] * reps
    inp = make(cuda_device, CHUNKS * reps, LENS * reps, 6, 2, 64, f16, seed=1, starts=starts,
               window=window)
    check(inp, 0.125, softcap=12.0)


@pytest.mark.gpu
@pytest.mark.parametrize("window,bias", [(0, False), (0, True), (64, False)])
@pytest.mark.parametrize("reps", [1, 8])
def test_prefixes(cuda_device, window, bias, reps):
    prefixes = [1, 60, 17, 2 ** 31 - 1, 64, 900, 380, 400, 9, -3] * reps
    starts = [0, 10, 3, 0, 70, 0, 390, 0, 0, 0] * reps
    inp = make(cuda_device, CHUNKS * reps, LENS * reps, 8, 2, 128, bf, seed=4, prefixes=prefixes,
               starts=starts, window=window)
    check(inp, 0.1, softcap=25.0, slopes=slopes_of(8, cuda_device) if bias else None)


@pytest.mark.gpu
def test_documents_share_one_cached_sequence(cuda_device):
    """Three documents packed into one cached sequence: three entries on one table
    row give what each document gives alone."""
    dev = cuda_device
    ends = [100, 333, 640]
    inp = make(dev, [640], [640], 8, 2, 64, bf, seed=7)
    docs = dict(inp, tables=inp["tables"] * 3, lens=ends, chunks=[100, 233, 307],
                starts=[0, 100, 333])
    check(docs, 0.125, softcap=30.0)


@pytest.mark.gpu
@pytest.mark.parametrize("scale,cap,q_std", [(1.0, 0.0, 30.0), (1.0, 50.0, 30.0), (-0.5, 8.0, 2.0),
                                             (-0.1, 0.0, 2.0), (0.0, 0.0, 1.0), (0.0, 4.0, 1.0),
                                             (0.1, 1e3, 2.0), (0.1, 1e6, 2.0), (0.1, 1e9, 2.0),
                                             (0.1, 1e15, 2.0), (0.1, 0.01, 2.0), (1e-4, 300.0, 1.0)])
def test_extreme_scores(cuda_device, scale, cap, q_std):
    inp = make(cuda_device, [100, 30], [100, 700], 8, 2, 128, bf, seed=9, q_std=q_std)
    check(inp, scale, softcap=cap)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [bf, f16])
@pytest.mark.parametrize("cap", [60.0, 40.0, 24.0, 12.0, 7.5, 6.0, 4.0])
@pytest.mark.parametrize("sign,bias", [(1, False), (-1, False), (1, True)])
def test_scores_at_every_share_of_the_cap(cuda_device, dtype, cap, sign, bias):
    """Largest scores from a sixth of the cap to several times it: tanh has a form for
    each range, chosen for a warp's scores at a time."""
    inp = make(cuda_device, [300, 130], [300, 700], 8, 2, 128, dtype, seed=11, q_std=2.0)
    check(inp, sign * 128 ** -0.5, softcap=cap, slopes=slopes_of(8, cuda_device) if bias else None)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,scale,cap", [(bf, 0.1, 1e6), (f16, 0.1, 1e5), (bf, 0.1, 50.0)])
@pytest.mark.parametrize("reps", [1, 30])
def test_large_scores_leave_small_ones_exact(cuda_device, dtype, scale, cap, reps):
    """Rows whose scores reach the cap beside rows whose scores are far below it, after
    a call that left huge values wherever the kernel keeps its tiles."""
    dev = cuda_device
    big = make(dev, [200] * 40, [300] * 40, 4, 2, 128, dtype, seed=1)
    big["k_cache"].fill_(3e4)
    big["v_cache"].fill_(-3e4)
    inp = make(dev, [100, 30] * reps, [100, 700] * reps, 8, 2, 128, dtype, seed=9, q_std=2.0)
    inp["q"][5::16] *= 0.9 * cap / (scale * 30.0) if cap < 1e3 else 2.0 ** 9
    run(big, 1.0, softcap=1e6)
    check(inp, scale, softcap=cap)


@pytest.mark.gpu
@pytest.mark.parametrize("reps", [1, 24])
def test_hidden_values_never_reach_a_row(cuda_device, reps):
    """Infinities and NaN in K and V of keys that some rows see and others do not:
    the rows that do not are what they would be without them."""
    dev = cuda_device
    inp = make(dev, [200, 60] * reps, [260, 300] * reps, 4, 2, 64, bf, seed=11, window=150)
    kc, vc = inp["k_cache"], inp["v_cache"]
    for s in range(2 * reps):
        for t, what in ((199, float("nan")), (250, float("inf")), (255, float("-inf"))):
            b = inp["tables"][s][t // 16]
            vc[b, t % 16, s % 2, 3 + t % 7] = what
        kc[inp["tables"][s][258 // 16], 258 % 16, 0, 9] = float("nan")
    check(inp, 0.125, softcap=20.0)


@pytest.mark.gpu
@pytest.mark.parametrize("reps", [1, 30])
def test_bad_table_entries_are_flagged_and_hidden(cuda_device, reps):
    inp = make(cuda_device, [50, 140] * reps, [300, 200] * reps, 4, 2, 128, f16, seed=8)
    NB = inp["k_cache"].shape[0]
    inp["tables"][0][2], inp["tables"][0][18], inp["tables"][1][0] = NB, -7, 2 ** 31 - 1
    check(inp, 0.1, softcap=9.0, flags=pkv.DEV_BAD_BLOCK_ID)


@pytest.mark.gpu
def test_bad_chunks_are_flagged_and_skipped(cuda_device):
    """A chunk longer than its context, than the bound, past the rows, or with a length
    past the table leaves its rows alone."""
    dev = cuda_device
    inp = make(dev, [20, 30, 10, 40], [100, 30, 60, 90], 4, 2, 64, bf, seed=3)
    for lens, cu, mx, dead in (([100, 29, 60, 90], [0, 20, 50, 60, 100], 40, 1),
                               ([100, 30, 60, 90], [0, 20, 50, 60, 100], 39, 3),
                               ([100, 30, 60, 90], [0, 20, 50, 60, 101], 41, 3),
                               ([100, 30, 113, 90], [0, 20, 50, 60, 100], 40, 2)):
        bad = dict(inp, lens=lens)
        out = run(bad, 0.125, flags=pkv.DEV_BAD_LENGTH, max_chunk=mx, cu=cu)
        want, tol = attention(inp["q"], inp["k_cache"], inp["v_cache"], inp["tables"],
                              inp["lens"], inp["chunks"], 0.125)
        at = [0, 20, 50, 60, 100]
        assert (out[at[dead]:at[dead + 1]] == 3.0).all()
        for s in range(4):
            if s != dead:
                sl = slice(at[s], at[s + 1])
                assert_close(out[sl], want[sl], tol[sl])


@pytest.mark.gpu
def test_one_row_chunks_match_the_decode_form(cuda_device):
    """The two forms agree on single tokens within their common bound."""
    dev = cuda_device
    lens = [1, 40, 129, 700, 2000]
    inp = make(dev, [1] * 5, lens, 8, 2, 128, bf, seed=6, window=600)
    sl = slopes_of(8, dev)
    a = run(inp, 0.1, 20.0, sl)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    out = torch.empty_like(inp["q"])
    pkv.paged_attention_decode_scored(
        inp["q"], inp["k_cache"], inp["v_cache"], i32(inp["tables"]), i32(lens), 2000, 0.1, out,
        pkv.new_scored_workspace(5, 8, 2, 128, 2000, dev), softcap=20.0, alibi_slopes=sl,
        window=600)
    want, tol = attention(inp["q"], inp["k_cache"], inp["v_cache"], inp["tables"], lens, None,
                          0.1, 20.0, sl, 600)
    assert_close(a, want, tol)
    assert_close(out, want, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("chunks,lens", [([5, 3], [700, 900]), ([300] * 12, [300, 700] * 6)])
def test_graph_replay_on_another_stream(cuda_device, chunks, lens):
    dev = cuda_device
    inp = make(dev, chunks, lens, 8, 2, 64, bf, seed=1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    cu = [sum(chunks[:i]) for i in range(len(chunks) + 1)]
    t = [i32(inp["tables"]), i32(lens), i32(cu)]
    out = torch.zeros_like(inp["q"])
    ws = pkv.new_prefill_scored_workspace(len(lens), max(chunks), 8, 2, 64, dev)
    call = lambda: pkv.paged_attention_prefill_scored(
        inp["q"], inp["k_cache"], inp["v_cache"], t[0], t[1], t[2], max(chunks), 0.125, out, ws,
        softcap=15.0)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    st = torch.cuda.Stream()
    shorter = [n - (n - c) // 2 for c, n in zip(chunks, lens)]
    for now in (lens, shorter):
        t[1].copy_(i32(now))
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for _ in range(5):
                graph.replay()
        torch.cuda.synchronize()
        want, tol = attention(inp["q"], inp["k_cache"], inp["v_cache"], inp["tables"], now,
                              chunks, 0.125, 15.0)
        assert_close(out, want, tol)
    first = out.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and pkv.pkv_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [f16, bf])
@pytest.mark.parametrize("cap", [0.0, 25.0])
def test_ragged_chunks_repeat_bit_for_bit(cuda_device, dtype, cap):
    """Items with and without a second tile in every order, sorted and dealt: equal
    calls give equal bits, and the bits of the definition's bound."""
    gen = torch.Generator().manual_seed(3)
    chunks = [int(x) for x in torch.randint(1, 420, (40,), generator=gen)]
    lens = [c + int(x) for c, x in zip(chunks, torch.randint(0, 900, (40,), generator=gen))]
    inp = make(cuda_device, chunks, lens, 10, 5, 128, dtype, seed=12, q_std=4.0)
    out = run(inp, 0.1, softcap=cap)
    for _ in range(15):
        assert torch.equal(run(inp, 0.1, softcap=cap), out)
    want, tol = attention(inp["q"], inp["k_cache"], inp["v_cache"], inp["tables"], lens, chunks,
                          0.1, cap)
    assert_close(out, want, tol)


@pytest.mark.gpu
def test_out_at_a_16_byte_address(cuda_device):
    """out and q may start at any 16-byte boundary."""
    dev = cuda_device
    inp = make(dev, [150, 7], [150, 600], 4, 2, 64, bf, seed=2)
    R = 157
    flat = torch.zeros(R * 4 * 64 + 8, dtype=bf, device=dev)
    qf = torch.zeros_like(flat)
    out, q = flat[8:].view(R, 4, 64), qf[8:].view(R, 4, 64)
    q.copy_(inp["q"])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    pkv.paged_attention_prefill_scored(
        q, inp["k_cache"], inp["v_cache"], i32(inp["tables"]), i32(inp["lens"]),
        i32([0, 150, 157]), 150, 0.125, out,
        pkv.new_prefill_scored_workspace(2, 150, 4, 2, 64, dev), softcap=10.0)
    want, tol = attention(inp["q"], inp["k_cache"], inp["v_cache"], inp["tables"], inp["lens"],
                          inp["chunks"], 0.125, 10.0)
    assert_close(out, want, tol)
