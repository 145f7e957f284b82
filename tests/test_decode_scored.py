"""Decode attention with capped and biased scores, windows and key starts,
against the definition in 64 bits; its refusals."""
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
    B, Hq, Hkv, D, NB = 3, 8, 2, 64, 10
    a = dict(q=torch.zeros(B, Hq, D, dtype=bf), k_cache=torch.zeros(NB, 16, Hkv, D, dtype=bf),
             v_cache=torch.zeros(NB, 16, Hkv, D, dtype=bf),
             block_tables=torch.zeros(B, 4, dtype=torch.int32),
             context_lens=torch.ones(B, dtype=torch.int32), max_context_len=64, scale=0.125,
             out=torch.zeros(B, Hq, D, dtype=bf), workspace=torch.zeros(1024, dtype=torch.uint8))
    a.update(over)
    return a


@pytest.mark.parametrize("over,msg", [
    (dict(alibi_slopes=torch.zeros(8, dtype=bf)), "alibi_slopes must be float32"),
    (dict(alibi_slopes=torch.zeros(2)), "alibi_slopes must be float32"),
    (dict(key_starts=torch.zeros(3, dtype=torch.int64)), "key_starts must be int32"),
    (dict(key_starts=torch.zeros(4, dtype=torch.int32)), "key_starts must be int32"),
    (dict(context_lens=torch.ones(2, dtype=torch.int32)), "context_lens must be int32"),
    (dict(out=torch.zeros(3, 8, 64, dtype=f16)), "share one dtype"),
    (dict(), "must be a CUDA tensor"),  # (the refusal that every well-formed call here meets)
])
def test_decode_scored_refuses(over, msg):
    with pytest.raises(ValueError, match=msg):
        pkv.paged_attention_decode_scored(**_cpu_args(**over))


def _c_call(entry="paged_attention_decode_scored", **over):
    a = dict(q=1 << 20, k_cache=2 << 20, v_cache=3 << 20, block_tables=4 << 20,
             max_blocks_per_seq=4, context_lens=5 << 20, max_context_len=64, num_seqs=2,
             num_q_heads=8, num_kv_heads=2, head_dim=64, num_blocks=8, scale=0.1, softcap=0.0,
             alibi_slopes=None, window=0, key_starts=None, out=6 << 20, workspace=7 << 20,
             workspace_bytes=1 << 30, dtype=1, stream=None)
    a.update(over)
    if entry.endswith("_packed"):
        slots = pkv._SLOTS[entry[:-7]](*(0 if v is None else v for v in a.values()))
        return getattr(pkv.lib(), entry)(slots)
    return pkv.lib().paged_attention_decode_scored(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(softcap=-1.0), 1),
    (dict(softcap=float("nan")), 1), (dict(softcap=1e-45, scale=1.0), 1), (dict(window=-1), 1),
    (dict(num_q_heads=9), 1), (dict(dtype=3), 1), (dict(num_seqs=-1), 1), (dict(q=None), 1),
    (dict(out=None), 1), (dict(q=(1 << 20) + 4), 1), (dict(max_context_len=-1), 1),
    (dict(num_q_heads=18), 2), (dict(head_dim=96), 2), (dict(num_seqs=8193), 2),
    (dict(max_blocks_per_seq=1 << 27), 2), (dict(num_blocks=1 << 27), 2),
    (dict(workspace=None), 6), (dict(workspace_bytes=1000), 6), (dict(workspace=(7 << 20) + 16), 6),
    (dict(num_seqs=0), 0), (dict(num_seqs=0, q=None, workspace=None), 0),
    (dict(out=1 << 20), 1), (dict(out=(1 << 20) + 2032), 1), (dict(out=(1 << 20) - 2032), 1),
])
def test_decode_scored_c_statuses(over, status):
    assert _c_call(**over) == status


@pytest.mark.parametrize("over", [{}, dict(q=None), dict(scale=float("nan")), dict(softcap=-1.0),
                                  dict(num_q_heads=18), dict(workspace_bytes=1000),
                                  dict(num_seqs=0), dict(dtype=3), dict(out=1 << 20)])
def test_packed_arguments_mean_the_same(over):
    """One array of 8-byte slots for the argument list."""
    base = dict(workspace_bytes=0)    # (a refusal either way: no kernel runs)
    packed = _c_call(entry="paged_attention_decode_scored_packed", **{**base, **over})
    assert packed == _c_call(**{**base, **over})


def test_packed_integers_are_not_cut():
    for name in ("num_seqs", "max_context_len", "window", "dtype", "workspace_bytes"):
        for wrong in (2 ** 32, -2 ** 32) if name != "workspace_bytes" else (-1,):
            # (cut to 32 bits the call would only find its workspace too small)
            assert _c_call(entry="paged_attention_decode_scored_packed",
                           **{"workspace_bytes": 1000, name: wrong}) == 1
    assert pkv.lib().paged_attention_decode_scored_packed(None) == 1


def test_workspace_size():
    f = pkv.paged_attention_decode_scored_workspace_bytes
    assert f(1, 8, 2, 96, 64) == 0 and f(0, 8, 2, 64, 64) == 0 and f(1, 8, 3, 64, 64) == 0
    assert 0 < f(8192, 64, 8, 128, 1 << 20) < 32 << 20


# ------------------------------------------------------------------ parity (GPU)
def make(dev, lens, Hq, Hkv, D, dtype, seed=0, q_std=1.5, starts=None, window=0, extra=5,
         max_blocks=None):
    """Inputs with every slot that holds no visible key poisoned with NaN, and table
    entries of blocks without a visible key set to -1."""
    g = torch.Generator(device=dev).manual_seed(seed)
    B = len(lens)
    need = [(max(n, 0) + BS - 1) // BS for n in lens]
    MB = max_blocks or max(max(need), 1)
    NB = sum(need) + extra
    perm = torch.randperm(NB, generator=g, device=dev).tolist()
    kc = torch.full((NB * BS, Hkv, D), float("nan"), dtype=dtype, device=dev)
    vc = torch.full((NB * BS, Hkv, D), float("nan"), dtype=dtype, device=dev)
    tables, at = [], 0
    for s, n in enumerate(lens):
        ids = perm[at:at + need[s]]
        at += need[s]
        lo = max(starts[s] if starts is not None else 0, 0, n - window if window else 0)
        if n > 0 and lo < n:
            t = torch.arange(lo, n, device=dev)
            slots = torch.tensor(ids, device=dev)[t // BS] * BS + t % BS
            kc[slots] = torch.randn(n - lo, Hkv, D, generator=g, device=dev).to(dtype)
            vc[slots] = torch.randn(n - lo, Hkv, D, generator=g, device=dev).to(dtype)
            ids = [-1] * (lo // BS) + ids[lo // BS:]
        else:
            ids = [-1] * len(ids)
        tables.append(ids + [-1] * (MB - need[s]))
    q = (torch.randn(B, Hq, D, generator=g, device=dev) * q_std).to(dtype)
    return dict(q=q, k_cache=kc.view(NB, BS, Hkv, D), v_cache=vc.view(NB, BS, Hkv, D),
                tables=tables, lens=list(lens), starts=starts, window=window)


def run(inp, max_len, scale, softcap=0.0, slopes=None, stream=None, ws=None, flags=0):
    dev = inp["q"].device
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=dev)
    B, Hq, D = inp["q"].shape
    Hkv = inp["k_cache"].shape[2]
    out = torch.full_like(inp["q"], 3.0)
    if ws is None:
        ws = pkv.new_scored_workspace(B, Hq, Hkv, D, max_len, dev).fill_(255)
    args = (i32(inp["tables"]), i32(inp["lens"]), i32(inp["starts"]))
    torch.cuda.synchronize()
    pkv.paged_attention_decode_scored(
        inp["q"], inp["k_cache"], inp["v_cache"], args[0], args[1], max_len, scale, out, ws,
        softcap=softcap, alibi_slopes=slopes, window=inp["window"], key_starts=args[2],
        stream=stream)
    torch.cuda.synchronize()
    assert pkv.pkv_device_status() == flags
    return out


def check(inp, max_len, scale, softcap=0.0, slopes=None, what="", **kw):
    out = run(inp, max_len, scale, softcap, slopes, **kw)
    want, tol = attention(inp["q"], inp["k_cache"], inp["v_cache"], inp["tables"], inp["lens"],
                          None, scale, softcap, slopes, inp["window"], inp["starts"])
    return assert_close(out, want, tol, what)


def slopes_of(Hq, dev):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / Hq) for i in range(Hq)], device=dev)


HEADS = [(1, 1, 64), (8, 8, 128), (16, 8, 128), (12, 4, 64), (8, 1, 128), (7, 1, 64), (15, 3, 64),
         (30, 6, 64), (32, 4, 64), (18, 3, 128)]
EDGE_LENS = [1, 2, 15, 16, 17, 31, 32, 33, 64, 100, 127, 128, 0, 5]
LONG_LENS = [1, 17, 128, 129, 500, 1000, 2047, 2048, 4100, 0, 16, 333]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [f16, bf])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("lens", [EDGE_LENS, LONG_LENS], ids=["rows", "split"])
def test_head_layouts_with_cap_and_bias(cuda_device, lens, Hq, Hkv, D, dtype):
    inp = make(cuda_device, lens, Hq, Hkv, D, dtype, seed=Hq + D)
    check(inp, max(lens), D ** -0.5, softcap=20.0, slopes=slopes_of(Hq, cuda_device))


@pytest.mark.gpu
@pytest.mark.parametrize("cap,bias", [(0.0, False), (0.0, True), (30.0, False), (5.0, True)])
@pytest.mark.parametrize("lens", [EDGE_LENS, LONG_LENS], ids=["rows", "split"])
@pytest.mark.parametrize("D", [64, 128])
def test_cap_and_bias(cuda_device, lens, cap, bias, D):
    inp = make(cuda_device, lens, 16, 4, D, f16, seed=3, q_std=4.0)
    check(inp, max(lens), D ** -0.5, softcap=cap,
          slopes=slopes_of(16, cuda_device) if bias else None)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 113, 114, 1000, 2 ** 31 - 1])
def test_windows(cuda_device, window):
    inp = make(cuda_device, LONG_LENS, 8, 2, 128, bf, seed=window % 1000, window=window)
    check(inp, 4100, 0.1, softcap=10.0, slopes=slopes_of(8, cuda_device))


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("lens,bound", [(EDGE_LENS, 128), (LONG_LENS, 4100)])
def test_key_starts_and_empty_rows(cuda_device, lens, bound, window):
    starts = [[0, -3, 14, 16, 17, 5, 40, 1, 63, 1 << 30, n - 1, -2 ** 31, 0, 4][i]
              for i, n in enumerate(lens)]
    inp = make(cuda_device, lens, 6, 3, 64, f16, seed=1, starts=starts, window=window)
    check(inp, bound, 0.125)
    inp = make(cuda_device, lens, 4, 2, 128, bf, seed=2, starts=list(lens), window=window)
    assert not run(inp, bound, 0.125).any()           # every row is empty


@pytest.mark.gpu
@pytest.mark.parametrize("B,n", [(1, 1), (1, 16), (1, 30000), (2, 9999), (700, 40), (3000, 33),
                                 (3000, 200), (8192, 17), (8192, 130)])
def test_batches(cuda_device, B, n):
    """One long sequence joined from every warp, and batches whose lengths leave two
    stages a warp."""
    lens = [max(1, n - (i * 7) % max(n // 2, 1)) for i in range(B)]
    Hq, Hkv = (8, 2) if B < 1000 else (2, 1)
    inp = make(cuda_device, lens, Hq, Hkv, 64 if B > 1000 else 128, bf, seed=B + n)
    if B <= 700:
        check(inp, n, 0.1, softcap=25.0)
        return
    out = run(inp, n, 0.1, softcap=25.0)
    pick = sorted({0, 1, B // 2, B - 1, *range(0, B, B // 40)})
    want, tol = attention(inp["q"][pick], inp["k_cache"], inp["v_cache"],
                          [inp["tables"][i] for i in pick], [lens[i] for i in pick], None, 0.1,
                          softcap=25.0)
    assert_close(out[pick], want, tol)
    assert torch.isfinite(out).all()


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv,D,window", [(8, 128, 0), (8, 64, 0), (3, 64, 20000)])
def test_long_batches(cuda_device, Hkv, D, window):
    """Long contexts in a batch, several sequences to a warp's run and several warps
    to a sequence: checked on some sequences, and the same from call to call."""
    B, g = 26 if Hkv == 8 else 40, 2
    lens = [40000 - 531 * i for i in range(B)]
    dev = cuda_device
    gen = torch.Generator(device=dev).manual_seed(5)
    need = [(n + BS - 1) // BS for n in lens]
    NB = sum(need)
    tables, at = [], 0
    perm = torch.randperm(NB, generator=gen, device=dev).tolist()
    for x in need:
        tables.append(perm[at:at + x] + [0] * (max(need) - x))
        at += x
    mk = lambda *s: torch.randn(*s, generator=gen, device=dev, dtype=torch.float32).to(f16)
    kc, vc = (torch.empty(NB, BS, Hkv, D, dtype=f16, device=dev) for _ in range(2))
    for i in range(0, NB, 4096):
        m = min(4096, NB - i)
        kc[i:i + m], vc[i:i + m] = mk(m, BS, Hkv, D), mk(m, BS, Hkv, D)
    inp = dict(q=mk(B, Hkv * g, D), k_cache=kc, v_cache=vc, tables=tables, lens=lens, starts=None,
               window=window)
    ws = pkv.new_scored_workspace(B, Hkv * g, Hkv, D, 40000, dev).fill_(255)
    out = run(inp, 40000, D ** -0.5, softcap=30.0, ws=ws)
    for s in (0, 1, B // 2, B - 1):
        want, tol = attention(inp["q"][s:s + 1], kc, vc, [tables[s]], [lens[s]], None, D ** -0.5,
                              softcap=30.0, window=window)
        assert_close(out[s:s + 1], want, tol)
    for _ in range(4):
        assert torch.equal(run(inp, 40000, D ** -0.5, softcap=30.0, ws=ws), out)


@pytest.mark.gpu
@pytest.mark.parametrize("scale,cap,q_std", [(1.0, 0.0, 30.0), (1.0, 50.0, 30.0), (-0.5, 8.0, 2.0),
                                             (0.0, 0.0, 1.0), (0.1, 1e3, 2.0), (0.1, 1e6, 2.0),
                                             (0.1, 1e9, 2.0), (0.1, 1e15, 2.0), (0.1, 0.01, 2.0),
                                             (1e-4, 300.0, 1.0)])
def test_extreme_scores(cuda_device, scale, cap, q_std):
    inp = make(cuda_device, [1, 50, 700], 8, 2, 128, bf, seed=9, q_std=q_std)
    check(inp, 700, scale, softcap=cap)


@pytest.mark.gpu
def test_negative_slopes_favour_far_keys(cuda_device):
    inp = make(cuda_device, [3, 300, 900], 4, 4, 64, bf, seed=4)
    check(inp, 900, 0.125, slopes=torch.tensor([-1.0, -0.01, 0.0, 0.5], device=cuda_device))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [100, 2000])
def test_bad_table_entries_are_flagged_and_hidden(cuda_device, n):
    inp = make(cuda_device, [n, n - 9], 8, 2, 128, f16, seed=8)
    NB = inp["k_cache"].shape[0]
    inp["tables"][0][2], inp["tables"][0][(n - 1) // 16], inp["tables"][1][0] = NB, -7, 2 ** 31 - 1
    check(inp, n, 0.1, softcap=9.0, flags=pkv.DEV_BAD_BLOCK_ID)


@pytest.mark.gpu
@pytest.mark.parametrize("bound", [100, 1000])
def test_bad_lengths_are_flagged_and_zero(cuda_device, bound):
    inp = make(cuda_device, [50, 70, 90, 60], 4, 2, 64, bf, seed=8)
    inp["lens"] = [50, bound + 1, -5, 60]
    out = run(inp, bound, 0.1, flags=pkv.DEV_BAD_LENGTH)
    assert not out[1:3].any()
    want, tol = attention(inp["q"], inp["k_cache"], inp["v_cache"], inp["tables"], [50, 0, 0, 60],
                          None, 0.1)
    assert_close(out, want, tol)


@pytest.mark.gpu
def test_non_finite_visible_values_follow_the_formula(cuda_device):
    """A NaN or infinity in a visible V element reaches that element of its group only."""
    inp = make(cuda_device, [40, 300], 4, 2, 64, bf, seed=5)
    blk = inp["tables"][1][3]
    inp["v_cache"][blk, 5, 1, 7] = float("nan")
    inp["v_cache"][blk, 6, 0, 9] = float("inf")
    out = run(inp, 300, 0.125)
    assert out[1, 2:, 7].isnan().all() and out[1, :2, 9].isinf().all()
    assert int((~torch.isfinite(out)).sum()) == 4


@pytest.mark.gpu
def test_graph_replay_and_streams(cuda_device):
    """Captured once, replayed with other lengths, starts and tables; two graphs with
    workspaces of their own replayed together on two streams."""
    dev = cuda_device
    cases = [make(dev, [300, 5, 1200, 64], 8, 2, 64, f16, seed=s, starts=[0, 2, 100, 0])
             for s in (1, 2)]
    sl = slopes_of(8, dev)
    graphs, outs, bufs = [], [], []
    for inp in cases:
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
        b = (i32(inp["tables"]), i32(inp["lens"]), i32(inp["starts"]))
        out = torch.zeros_like(inp["q"])
        ws = pkv.new_scored_workspace(4, 8, 2, 64, 1200, dev)
        call = lambda: pkv.paged_attention_decode_scored(
            inp["q"], inp["k_cache"], inp["v_cache"], b[0], b[1], 1200, 0.125, out, ws,
            softcap=15.0, alibi_slopes=sl, key_starts=b[2])
        call()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call()
        graphs.append(gr)
        outs.append(out)
        bufs.append((b, ws))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for lens, starts in (([300, 5, 1200, 64], [0, 2, 100, 0]), ([170, 3, 1111, 1], [160, 2, 1000, 1])):
        for (b, _), out in zip(bufs, outs):
            b[1].copy_(torch.tensor(lens, dtype=torch.int32))
            b[2].copy_(torch.tensor(starts, dtype=torch.int32))
            out.fill_(9.0)
        torch.cuda.synchronize()
        for _ in range(20):
            for st, gr in zip(streams, graphs):
                with torch.cuda.stream(st):
                    gr.replay()
        torch.cuda.synchronize()
        for inp, out in zip(cases, outs):
            want, tol = attention(inp["q"], inp["k_cache"], inp["v_cache"], inp["tables"], lens,
                                  None, 0.125, 15.0, sl, 0, starts)
            assert_close(out, want, tol)
    assert pkv.pkv_device_status() == 0


@pytest.mark.gpu
def test_results_do_not_change_from_call_to_call(cuda_device):
    inp = make(cuda_device, LONG_LENS, 16, 8, 128, bf, seed=6)
    first = run(inp, 4100, 0.1, softcap=30.0)
    for _ in range(5):
        assert torch.equal(run(inp, 4100, 0.1, softcap=30.0), first)


@pytest.mark.gpu
def test_pools_past_two_to_the_31_elements(cuda_device):
    dev = cuda_device
    Hkv, D, NB = 8, 128, (1 << 31) // (BS * 8 * 128) + 50
    n = 700
    kc = torch.zeros(NB, BS, Hkv, D, dtype=bf, device=dev)
    vc = torch.zeros(NB, BS, Hkv, D, dtype=bf, device=dev)
    ids = [NB - 1 - i if i % 2 else i for i in range((n + BS - 1) // BS)]
    at = torch.tensor(ids, device=dev)
    kc[at] = torch.randn(len(ids), BS, Hkv, D, device=dev).to(bf)
    vc[at] = torch.randn(len(ids), BS, Hkv, D, device=dev).to(bf)
    inp = dict(q=torch.randn(1, 16, D, device=dev).to(bf), k_cache=kc, v_cache=vc, tables=[ids],
               lens=[n], starts=None, window=0)
    check(inp, n, 0.1, softcap=20.0)


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv,D", [(1, 128), (2, 64), (40, 64)])
def test_parts_whose_scores_are_all_minus_infinity(cuda_device, Hkv, D):
    """Keys that are seen with a score of -inf weigh nothing, whole parts of them in
    front of a far lower but finite maximum too: as though the keys started later."""
    lens = [2900, 2500, 700, 1] + [90] * 8
    inp = make(cuda_device, lens, 2 * Hkv, Hkv, D, f16, seed=D + Hkv)
    inp["q"][:, :, 0] = 4.0
    later = []
    for s, n in enumerate(lens):
        later.append(n * 2 // 3)
        for t in range(0, n, BS):
            block = inp["k_cache"][inp["tables"][s][t // BS]]
            block[:, :, 0] = -600.0
            block[:max(0, min(BS, later[-1] - t)), :, 0] = -float("inf")
    got = run(inp, 2900, 0.125)
    want, tol = attention(inp["q"], inp["k_cache"], inp["v_cache"], inp["tables"], lens, None, 0.125,
                          starts=later)
    assert_close(got, want, tol)
