"""The rotary write and the two attentions with modified scores used together, as a
serving loop uses them: a prompt in two chunks, then decode steps as one graph."""
import pytest
import torch

import paged_kv_cache_211_gb300 as pkv
from rope_reference import rotate
from scored_reference import assert_close, attention

BS = 16


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,R,interleaved,window", [
    (torch.bfloat16, 128, 128, False, 0), (torch.float16, 64, 32, True, 60),
])
def test_prompt_then_decode(cuda_device, dtype, D, R, interleaved, window):
    dev = cuda_device
    B, Hq, Hkv, layers = 3, 8, 2, 2
    prompts, steps, cap, scale = [70, 33, 150], 6, 20.0, D ** -0.5
    MB = (max(prompts) + steps + BS - 1) // BS
    NB = B * MB + 2
    g = torch.Generator(device=dev).manual_seed(D)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev).to(dtype)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    alloc = pkv.BlockAllocator(NB)
    tables = [alloc.alloc(MB) for _ in range(B)]
    bt = i32(tables)
    freq, m = pkv.paged_kv_rope_frequencies(R, scaling="yarn", factor=4.0,
                                            original_max_position=64, device=dev)
    kc = torch.full((layers, NB, BS, Hkv, D), float("nan"), dtype=dtype, device=dev)
    vc = torch.full_like(kc, float("nan"))
    slopes = torch.tensor([2.0 ** -(i + 1) for i in range(Hq)], device=dev)
    mods = dict(softcap=cap, alibi_slopes=slopes, window=window)

    # what the definition says: every token's unrotated rows, kept on the side
    hist = [[[] for _ in range(B)] for _ in range(layers)]    # (k, v) per layer and sequence

    def expect(layer, q64, lens, chunks):
        """Attention of the definition over rotated, rounded keys (the cache's type)."""
        K = torch.zeros(B * MB, BS, Hkv, D, dtype=dtype, device=dev)
        V = torch.zeros_like(K)
        for s in range(B):
            ks = torch.cat([k for k, _ in hist[layer][s]])
            vs = torch.cat([v for _, v in hist[layer][s]])
            n = lens[s]
            pos = list(range(n))
            rk = torch.tensor(rotate(ks.double().cpu().numpy(), pos, freq.cpu().numpy(), m,
                                     interleaved)[0], device=dev).to(dtype)
            K[s * MB:(s + 1) * MB].view(-1, Hkv, D)[:n] = rk
            V[s * MB:(s + 1) * MB].view(-1, Hkv, D)[:n] = vs
        pos = [n - c + i for n, c in zip(lens, chunks) for i in range(c)]
        rq = torch.tensor(rotate(q64, pos, freq.cpu().numpy(), m, interleaved)[0],
                          device=dev).to(dtype)
        want, tol = attention(rq, K, V, [list(range(s * MB, (s + 1) * MB)) for s in range(B)],
                              lens, chunks, scale, cap, slopes, window)
        # q and the keys are rounded twice the same way, except where the kernel's
        # and the definition's angles put a value on either side of a rounding
        # border: one step eps of such an element of q or k moves a score by at
        # most eps * scale * m * sum |q k| over a few of the D elements (4 of them
        # allowed for here, of 10 each), in base e; weights by twice that
        flip = 2 * torch.finfo(dtype).eps * scale * 4 * 10.0
        return want, tol + flip * want.abs().amax()

    # ---- the prompts in two chunks each, all layers
    done = [0] * B
    for part in (0.6, 1.0):
        chunks = [int(n * part) - d for n, d in zip(prompts, done)]
        lens = [d + c for d, c in zip(done, chunks)]
        rows = sum(chunks)
        pos, slots = [], []
        for s in range(B):
            for p in range(done[s], lens[s]):
                pos.append(p)
                slots.append(tables[s][p // BS] * BS + p % BS)
        cu = [0]
        for c in chunks:
            cu.append(cu[-1] + c)
        for layer in range(layers):
            qkv = rnd(rows, (Hq + 2 * Hkv) * D)
            q = qkv[:, :Hq * D].view(rows, Hq, D)
            k = qkv[:, Hq * D:(Hq + Hkv) * D].view(rows, Hkv, D)
            v = qkv[:, (Hq + Hkv) * D:].view(rows, Hkv, D)
            qr, out = torch.empty(rows, Hq, D, dtype=dtype, device=dev), None
            pkv.paged_kv_rope_write(q, k, v, kc[layer], vc[layer], i32(pos),
                                    torch.tensor(slots, device=dev), freq, qr,
                                    interleaved=interleaved, rope_scale=m)
            out = torch.empty_like(qr)
            ws = pkv.new_prefill_scored_workspace(B, max(chunks), Hq, Hkv, D, dev)
            pkv.paged_attention_prefill_scored(qr, kc[layer], vc[layer], bt, i32(lens), i32(cu),
                                               max(chunks), scale, out, ws, **mods)
            for s in range(B):
                hist[layer][s].append((k[cu[s]:cu[s + 1]].clone(), v[cu[s]:cu[s + 1]].clone()))
            want, tol = expect(layer, q.double().cpu().numpy(), lens, chunks)
            assert_close(out, want, tol, f"chunk to {part} layer {layer}")
        done = lens

    # ---- decode: one graph of every layer's write and attention, replayed per step
    qkv = torch.zeros(layers, B, (Hq + 2 * Hkv) * D, dtype=dtype, device=dev)
    cl = i32(done)
    qr = torch.zeros(layers, B, Hq, D, dtype=dtype, device=dev)
    out = torch.zeros_like(qr)
    ws = pkv.new_scored_workspace(B, Hq, Hkv, D, MB * BS, dev)

    def step():
        cl.add_(1)
        for layer in range(layers):
            x = qkv[layer]
            pkv.paged_kv_rope_write_new_tokens(
                x[:, :Hq * D].view(B, Hq, D), x[:, Hq * D:(Hq + Hkv) * D].view(B, Hkv, D),
                x[:, (Hq + Hkv) * D:].view(B, Hkv, D), kc[layer], vc[layer], bt, cl, freq,
                qr[layer], interleaved=interleaved, rope_scale=m)
            pkv.paged_attention_decode_scored(qr[layer], kc[layer], vc[layer], bt, cl, MB * BS,
                                              scale, out[layer], ws, **mods)

    step()                      # warm-up outside the graph, then taken back
    torch.cuda.synchronize()
    cl.sub_(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        qkv.copy_(rnd(layers, B, (Hq + 2 * Hkv) * D))
        graph.replay()
        torch.cuda.synchronize()
        lens = [n + i + 1 for n in prompts]
        for layer in range(layers):
            x = qkv[layer]
            k = x[:, Hq * D:(Hq + Hkv) * D].view(B, 1, Hkv, D)
            v = x[:, (Hq + Hkv) * D:].view(B, 1, Hkv, D)
            for s in range(B):
                hist[layer][s].append((k[s].clone(), v[s].clone()))
            want, tol = expect(layer, x[:, :Hq * D].view(B, Hq, D).double().cpu().numpy(), lens,
                               [1] * B)
            assert_close(out[layer], want, tol, f"step {i} layer {layer}")
    assert pkv.pkv_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("graph", [False, True])
def test_calls_in_a_row_see_one_another(cuda_device, graph):
    """Each call reads what the one in front of it wrote, and kernels are scheduled
    before their predecessors end: the same bits as with a wait after every call."""
    dev, dtype = cuda_device, torch.bfloat16
    B, Hq, Hkv, D, n, rounds = 4, 4, 2, 128, 900, 12
    MB = (n + BS - 1) // BS
    gen = torch.Generator(device=dev).manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev).to(dtype)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    bt = torch.randperm(B * MB, generator=gen, device=dev).to(torch.int32).view(B, MB)
    k0, v0, x0 = rnd(B * MB, BS, Hkv, D), rnd(B * MB, BS, Hkv, D), rnd(B, Hq, D)
    lens, cu = i32([n, n - 1, n - 40, n]), i32(range(B + 1))
    freq = pkv.paged_kv_rope_frequencies(D, device=dev)[0]
    ws = [pkv.new_scored_workspace(B, Hq, Hkv, D, n, dev),
          pkv.new_prefill_scored_workspace(B, 1, Hq, Hkv, D, dev),
          pkv.new_workspace(B, Hq, D, n, dev)]
    kc, vc, x = k0.clone(), v0.clone(), x0.clone()
    qr, a, b = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)

    def chain(after):
        for _ in range(rounds):
            pkv.paged_kv_rope_write_new_tokens(x, x[:, :Hkv], x[:, Hkv:], kc, vc, bt, lens, freq, qr)
            after()
            pkv.paged_attention_decode_scored(qr, kc, vc, bt, lens, n, 0.3, a, ws[0], softcap=90.0)
            after()
            pkv.paged_attention_prefill_scored(a, kc, vc, bt, lens, cu, 1, 0.3, b, ws[1],
                                               window=500)
            after()
            pkv.paged_attention_decode(b, kc, vc, bt, lens, n, 0.3, a, ws[2])
            after()
            pkv.paged_attention_prefill_scored(a, kc, vc, bt, lens, cu, 1, 0.3, b, ws[1],
                                               softcap=50.0)
            after()
            x.copy_(b * 8)
            after()

    def reset():
        for t, t0 in ((kc, k0), (vc, v0), (x, x0)):
            t.copy_(t0)
        torch.cuda.synchronize()

    chain(torch.cuda.synchronize)
    want = [t.clone() for t in (kc, vc, x, a, b, qr)]
    assert torch.isfinite(want[2]).all()
    reset()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            chain(lambda: None)
    for _ in range(5):
        reset()
        if graph:
            g.replay()
        else:
            chain(lambda: None)
        torch.cuda.synchronize()
        for t, w in zip((kc, vc, x, a, b, qr), want):
            assert torch.equal(t, w)
    assert pkv.pkv_device_status() == 0
