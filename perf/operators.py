"""Cases of the operators for models with rotary positions and modified attention scores.

Three operators over a block-paged KV cache (16-token blocks, pools [blocks, 16, kv heads, head dim]):

rope     rotary positions applied to q and k, and the write of the rotated k and of v into the cache:
         for packed tokens with positions and slots ("tokens"), or for one new token per sequence ("step");
decode   attention of one query per sequence, prefill: of a packed chunk of queries per sequence, with
         z = scale <q, k_t>, then cap * tanh(z / cap), then - slope |p - t| for the query at position p,
         over the keys max(0, key start, p - window + 1) <= t < max(p + 1, min(prefix length, length)).

Every case is a dict of plain values; `prepare` makes its inputs from the seed, `run` makes one pass in the
plain form (`own` false) or by the package's kernels (`own` true), and `exact` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

BS = 16  # tokens per cache block
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------- cases
def listed():
    """The measured cases; lengths within a case are drawn from its own "shape" number."""
    return [
        # one decode step's new tokens of a four-sequence batch: launch latency
        rope("rope_step_4seqs", "step", 4, 16, 8, 128, 128, "f16", lo=17, hi=100, shape=1),
        # one decode step of a large batch, grouped heads, 64-wide heads rotated in half of their width
        rope("rope_step_256seqs_partial", "step", 256, 32, 4, 64, 32, "f16", lo=1, hi=2048, shape=2,
             interleaved=True),
        # eight 2048-token prompts, the positions far out in a context stretched by YaRN's factors
        rope("rope_prompts_16384", "tokens", 16384, 32, 8, 128, 128, "bf16", lo=100000, hi=1000000, shape=3,
             scaling="yarn"),
        # a ragged batch of chunks, q, k and v as views of one projection's rows, padding tokens among them
        rope("rope_ragged_1777_packed", "tokens", 1777, 16, 4, 64, 48, "bf16", lo=0, hi=32768, shape=4,
             interleaved=True, packed=True, pad=13, scaling="linear"),
        # four short sequences with capped scores: latency
        decode("decode_4seqs_cap", 4, 16, 8, 128, "f16", 17, 100, shape=5, softcap=30.0),
        # a batch of short contexts with a distance bias, two padding rows behind it
        decode("decode_62rows_bias", 62, 16, 8, 128, "f16", 32, 512, shape=6, bias=True, pad=2),
        # long contexts of a 7B-shaped model with capped scores
        decode("decode_32seqs_long_cap", 32, 32, 8, 128, "bf16", 2048, 32768, shape=7, softcap=50.0, q_std=3.0),
        # a sliding window of 1000 tokens over 256 sequences
        decode("decode_256seqs_window", 256, 32, 4, 64, "f16", 600, 2048, shape=8, window=1000, softcap=50.0),
        # a few new tokens (drafted ones to verify) over middling contexts, capped: latency
        prefill("prefill_4seqs_draft_cap", 4, 16, 8, 128, "f16", 3, 8, 100, 2000, shape=9, softcap=30.0),
        # eight whole prompts of 2048 tokens with capped scores
        prefill("prefill_8x2048_cap", 8, 32, 8, 128, "bf16", 2048, 2048, 0, 0, shape=10, softcap=50.0, q_std=2.0),
        # ragged chunks with a window and a distance bias, grouped by three
        prefill("prefill_ragged_window_bias", 24, 12, 4, 64, "bf16", 1, 700, 0, 3000, shape=11, window=513,
                bias=True),
        # prompts whose prefix is seen from both sides, keys of an earlier document hidden
        prefill("prefill_prefix_documents", 12, 16, 2, 128, "f16", 100, 1500, 0, 500, shape=12, prefix=0.4,
                starts=True, softcap=20.0),
    ]


def rope(name, form, tokens, hq, hkv, d, rot, dtype, lo, hi, shape, interleaved=False, packed=False, pad=0,
         scaling="none"):
    return {"name": name, "op": "rope", "form": form, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "dtype": dtype, "lo": lo, "hi": hi, "shape": shape, "interleaved": interleaved, "packed": packed,
            "pad": pad, "scaling": scaling}


def decode(name, seqs, hq, hkv, d, dtype, lo, hi, shape, softcap=0.0, bias=False, window=0, starts=False, pad=0,
           q_std=1.5):
    return {"name": name, "op": "decode", "seqs": seqs, "hq": hq, "hkv": hkv, "d": d, "dtype": dtype, "lo": lo,
            "hi": hi, "shape": shape, "softcap": softcap, "bias": bias, "window": window, "starts": starts,
            "pad": pad, "q_std": q_std}


def prefill(name, seqs, hq, hkv, d, dtype, qlo, qhi, plo, phi, shape, softcap=0.0, bias=False, window=0,
            starts=False, prefix=0.0, q_std=1.5):
    return {"name": name, "op": "prefill", "seqs": seqs, "hq": hq, "hkv": hkv, "d": d, "dtype": dtype,
            "qlo": qlo, "qhi": qhi, "plo": plo, "phi": phi, "shape": shape, "softcap": softcap, "bias": bias,
            "window": window, "starts": starts, "prefix": prefix, "q_std": q_std}


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm where the range spans more than a factor of ten."""
    if hi <= lo:
        return lo
    if hi > 10 * max(lo, 1):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))))
    return rng.randint(lo, hi)


def draw(rng):
    """One more case of the ranges behind the listed ones, no dearer than the dearest of its operator."""
    op = rng.choice(["rope", "decode", "prefill"])
    top = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        d = rng.choice([64, 128])
        dtype = rng.choice(["f16", "bf16"])
        hkv = rng.choice([1, 2, 3, 4, 5, 8])
        group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
        shape = rng.randrange(1 << 30)
        cap = rng.choice([0.0, rng.uniform(5.0, 60.0)])
        bias = rng.random() < 0.4
        window = rng.choice([0, 0, _spread(rng, 1, 4000)])
        starts = rng.random() < 0.3
        if op == "rope":
            form = rng.choice(["step", "tokens"])
            tokens = _spread(rng, 1, 512 if form == "step" else 16384)
            lo = _spread(rng, 1, 1000)
            hi = lo + _spread(rng, 1, 2000 if form == "step" else 1000000)
            c = rope("", form, tokens, hkv * group, hkv, d, 2 * _spread(rng, 4, d // 2), dtype, lo, hi, shape,
                     rng.random() < 0.5, rng.random() < 0.5, rng.choice([0, 0, rng.randint(2, 20)]),
                     rng.choice(["none", "linear", "ntk", "yarn"]))
        elif op == "decode":
            lo = _spread(rng, 1, 8000)
            c = decode("", _spread(rng, 1, 300), hkv * group, hkv, d, dtype, lo, lo + _spread(rng, 1, 24000), shape,
                       cap, bias, window, starts, rng.choice([0, 0, 3]), rng.uniform(0.5, 4.0))
        else:
            qlo, plo = _spread(rng, 1, 500), rng.choice([0, _spread(rng, 1, 1000)])
            c = prefill("", _spread(rng, 1, 40), hkv * group, hkv, d, dtype, qlo, qlo + _spread(rng, 1, 1500), plo,
                        plo + _spread(rng, 1, 3000), shape, cap, bias, window, starts,
                        rng.choice([0.0, 0.0, rng.uniform(0.1, 0.9)]), rng.uniform(0.5, 3.0))
        del c["name"]
        if _cost(c) <= top:
            return c


def _lens(case):
    """Host lengths of an attention case, the same for every seed:
    decode: context lengths; prefill: (chunk lengths, context lengths, prefix lengths); both: key starts."""
    rng = random.Random(case["shape"])
    if case["op"] == "decode":
        n = [_spread(rng, case["lo"], case["hi"]) for _ in range(case["seqs"] - case["pad"])] + [0] * case["pad"]
        starts = [rng.randint(0, max(0, x - 1)) // 2 if case["starts"] else 0 for x in n]
        return n, starts
    q = [_spread(rng, case["qlo"], case["qhi"]) for _ in range(case["seqs"])]
    n = [x + _spread(rng, case["plo"], case["phi"]) for x in q]
    starts = [rng.randint(0, x) // 3 if case["starts"] else 0 for x in n]
    return q, n, [int(x * case["prefix"]) for x in n], starts


def _range(case, p, n, start, prefix=0):
    """The visible keys [lo, hi) of the query at position p of a sequence of n tokens."""
    lo = max(0, start, p - case["window"] + 1 if case["window"] else 0)
    return lo, max(p + 1, min(prefix, n))


def _tokens(case):
    """Host positions and padding marks of a rope case (the last padding tokens of a batch, or every pad-th)."""
    rng = random.Random(case["shape"])
    pos = [_spread(rng, case["lo"], case["hi"]) for _ in range(case["tokens"])]
    return pos, [bool(case["pad"]) and t % case["pad"] == 0 for t in range(case["tokens"])]


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        live = sum(not x for x in _tokens(case)[1])
        return {"bytes": live * (4 * (hq + 2 * hkv) * d + 12) + 2 * case["rot"],
                "flops": live * (hq + hkv) * case["rot"] * 3}
    rows = keys = pairs = 0
    if case["op"] == "decode":
        for n, start in zip(*_lens(case)):
            rows += 1
            lo, hi = _range(case, n - 1, n, start) if n else (0, 0)
            keys += max(0, hi - lo)
            pairs += max(0, hi - lo)
    else:
        for q, n, prefix, start in zip(*_lens(case)):
            rows += q
            spans = [_range(case, p, n, start, prefix) for p in range(n - q, n)]
            pairs += sum(max(0, hi - lo) for lo, hi in spans)
            keys += max(0, max(hi for _, hi in spans) - spans[0][0])
    return {"bytes": 4 * keys * hkv * d + 4 * rows * hq * d + 4 * (keys // BS) + 8 * case["seqs"],
            "flops": 4 * pairs * hq * d}


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1e15


# --------------------------------------------------------------------------- inputs
def _frequencies(case):
    """The rotary frequencies (fp32, on the host) and the factor on cos and sin of a case's context scaling."""
    rot, base, factor = case["rot"], 10000.0, 8.0
    e = torch.arange(0, rot, 2, dtype=torch.float64) / rot
    if case["scaling"] == "ntk":
        base = base * factor ** (rot / (rot - 2)) if rot > 2 else base
    f = base ** -e
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "yarn":  # original length 4096, ramp between 32 and 1 turns
        dim = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
    return f.float(), 0.1 * math.log(factor) + 1.0 if case["scaling"] == "yarn" else 1.0


def _table(lens, rng_perm, blocks):
    """Block tables of contexts that own their blocks, taken from a permutation of the pool."""
    width = max(1, max((n + BS - 1) // BS for n in lens))
    rows, at = [], 0
    for n in lens:
        need = (n + BS - 1) // BS
        rows.append(rng_perm[at:at + need] + [0] * (width - need))
        at += need
    assert at <= blocks
    return rows


def _inputs(case, seed):
    """Everything of a case that comes from the seed: q, k, v, pools, tables, lengths, on the GPU."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES[case["dtype"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]

    def normal(*shape, std=1.0):
        x = torch.empty(shape, dtype=dt, device=dev)
        flat = x.view(-1)
        for i in range(0, flat.numel(), 1 << 27):
            n = min(1 << 27, flat.numel() - i)
            flat[i:i + n] = torch.randn(n, generator=gen, device=dev) * std
        return x

    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    s = {"case": case}
    if case["op"] == "rope":
        t = case["tokens"]
        pos, pad = _tokens(case)
        if case["packed"]:
            rows = normal(t, (hq + 2 * hkv) * d)
            s["q"] = rows[:, :hq * d].view(t, hq, d)
            s["k"] = rows[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
            s["v"] = rows[:, (hq + hkv) * d:].view(t, hkv, d)
        else:
            s["q"], s["k"], s["v"] = normal(t, hq, d), normal(t, hkv, d), normal(t, hkv, d)
        freq, s["factor"] = _frequencies(case)
        s["freq"] = freq.to(dev)
        if case["form"] == "step":
            lens = [0 if x else p for p, x in zip(pos, pad)]
            blocks = max(1, sum((n + BS - 1) // BS for n in lens))
            table = _table(lens, rng.sample(range(blocks), blocks), blocks)
            slots = [table[i][(n - 1) // BS] * BS + (n - 1) % BS if n else -1 for i, n in enumerate(lens)]
            s["table"], s["lens"] = ints(table), ints(lens)
            pos = [max(n - 1, 0) for n in lens]
        else:
            blocks = (t + BS - 1) // BS + 1
            order = rng.sample(range(blocks), blocks)
            slots = [-1 if x else order[i // BS] * BS + i % BS for i, x in enumerate(pad)]
        s["k_cache"], s["v_cache"] = normal(blocks, BS, hkv, d), normal(blocks, BS, hkv, d)
        s["pos"] = ints(pos)
        s["slots"] = torch.tensor(slots, dtype=torch.int64, device=dev)
        s["live"] = torch.tensor([i for i, x in enumerate(slots) if x >= 0], dtype=torch.int64, device=dev)
        s["out"] = torch.zeros(t, hq, d, dtype=dt, device=dev)
        return s
    if case["op"] == "decode":
        lens, starts = _lens(case)
        rows = case["seqs"]
    else:
        s["chunks"], lens, prefix, starts = _lens(case)
        rows = sum(s["chunks"])
        cu = [0]
        for x in s["chunks"]:
            cu.append(cu[-1] + x)
        s["cu"] = ints(cu)
        s["prefix"] = ints(prefix) if case["prefix"] else None
        s["prefix_host"] = prefix
    blocks = max(1, sum((n + BS - 1) // BS for n in lens))
    s["lens_host"], s["starts_host"] = lens, starts
    s["table"] = ints(_table(lens, rng.sample(range(blocks), blocks), blocks))
    s["lens"] = ints(lens)
    s["starts"] = ints(starts) if case["starts"] else None
    s["k_cache"], s["v_cache"] = normal(blocks, BS, hkv, d), normal(blocks, BS, hkv, d)
    s["q"] = normal(rows, hq, d, std=case["q_std"])
    s["scale"] = d ** -0.5
    # slopes as a geometric row over the heads, as a distance bias is set up
    s["slopes"] = (torch.tensor([2.0 ** (-8.0 * (i + 1) / hq) for i in range(hq)], device=dev)
                   if case["bias"] else None)
    s["out"] = torch.empty_like(s["q"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"] != "rope":
        import paged_kv_cache_211_gb300 as pkv
        s["max_len"] = max(s["lens_host"] + [1])
        if case["op"] == "decode":
            s["workspace"] = pkv.new_scored_workspace(case["seqs"], case["hq"], case["hkv"], case["d"],
                                                      s["max_len"], s["q"].device)
        else:
            s["max_chunk"] = max(s["chunks"])
            s["workspace"] = pkv.new_prefill_scored_workspace(case["seqs"], s["max_chunk"], case["hq"], case["hkv"],
                                                              case["d"], s["q"].device)
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    return _plain_rope(s, case) if case["op"] == "rope" else _plain_attention(s, case)


def _run_own(s, case):
    import paged_kv_cache_211_gb300 as pkv
    if case["op"] == "rope":
        if case["form"] == "step":
            pkv.paged_kv_rope_write_new_tokens(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"],
                                               s["lens"], s["freq"], s["out"], interleaved=case["interleaved"],
                                               rope_scale=s["factor"])
        else:
            pkv.paged_kv_rope_write(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["pos"], s["slots"],
                                    s["freq"], s["out"], interleaved=case["interleaved"], rope_scale=s["factor"])
        return s["out"], s["k_cache"], s["v_cache"]
    if case["op"] == "decode":
        return pkv.paged_attention_decode_scored(
            s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["max_len"], s["scale"], s["out"],
            s["workspace"], softcap=case["softcap"], alibi_slopes=s["slopes"], window=case["window"],
            key_starts=s["starts"])
    return pkv.paged_attention_prefill_scored(
        s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"], s["max_chunk"], s["scale"], s["out"],
        s["workspace"], softcap=case["softcap"], alibi_slopes=s["slopes"], window=case["window"],
        key_starts=s["starts"], prefix_lens=s["prefix"])


def _plain_rope(s, case):
    """Angles in 64 bits (positions reach millions), the rotation in 32, one rounding; padding tokens untouched."""
    live, rot, half = s["live"], case["rot"], case["rot"] // 2
    angle = s["pos"][live].double()[:, None] * s["freq"].double()
    cos = (angle.cos() * s["factor"]).float()[:, None, :]
    sin = (angle.sin() * s["factor"]).float()[:, None, :]

    def turn(x):
        y = x[live].float()
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if case["interleaved"] else (y[..., :half], y[..., half:rot])
        c, e = a * cos - b * sin, b * cos + a * sin
        front = torch.stack((c, e), dim=-1).flatten(-2) if case["interleaved"] else torch.cat((c, e), dim=-1)
        return torch.cat((front, y[..., rot:]), dim=-1).to(x.dtype)

    slots = s["slots"][live]
    s["out"][live] = turn(s["q"])
    s["k_cache"].view(-1, case["hkv"], case["d"])[slots] = turn(s["k"])
    s["v_cache"].view(-1, case["hkv"], case["d"])[slots] = s["v"][live]
    return s["out"], s["k_cache"], s["v_cache"]


def _plain_attention(s, case):
    """Sequence by sequence in 32 bits: gather, scores, cap, bias, mask, softmax, weighted sum."""
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    out = s["out"]
    at = 0
    for i, n in enumerate(s["lens_host"]):
        rows = s["chunks"][i] if case["op"] == "prefill" else 1
        here, at = slice(at, at + rows), at + rows
        start = s["starts_host"][i]
        prefix = s["prefix_host"][i] if case["op"] == "prefill" else 0
        lo, _ = _range(case, n - rows, n, start)
        _, hi = _range(case, n - 1, n, start, prefix)
        if n == 0 or lo >= hi:
            out[here] = 0
            continue
        ids = s["table"][i, lo // BS:(hi + BS - 1) // BS].long()
        cut = slice(lo % BS, lo % BS + hi - lo)
        k = s["k_cache"][ids].view(-1, hkv, d)[cut].float().permute(1, 2, 0)      # hkv, d, keys
        v = s["v_cache"][ids].view(-1, hkv, d)[cut].float().permute(1, 0, 2)      # hkv, keys, d
        q = s["q"][here].float().view(rows, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, g * rows, d)
        z = torch.matmul(q, k).view(hkv, g, rows, hi - lo) * s["scale"]
        if case["softcap"]:
            z = torch.tanh(z / case["softcap"]) * case["softcap"]
        t = torch.arange(lo, hi, device=q.device)
        p = torch.arange(n - rows, n, device=q.device)[:, None]
        if s["slopes"] is not None:
            z = z - s["slopes"].view(hkv, g, 1, 1) * (p - t).abs().float()
        seen = (t >= start) & ((t <= p) | (t < prefix))
        if case["window"]:
            seen = seen & (t > p - case["window"])
        z = z.masked_fill(~seen, float("-inf"))
        top = z.amax(dim=-1, keepdim=True)
        e = torch.exp(z - torch.where(top == float("-inf"), torch.zeros_like(top), top))
        total = e.sum(dim=-1, keepdim=True)
        w = e / torch.where(total == 0, torch.ones_like(total), total)
        o = torch.matmul(w.view(hkv, g * rows, hi - lo), v).view(hkv, g, rows, d)
        out[here] = o.permute(2, 0, 1, 3).reshape(rows, hq, d).to(out.dtype)
    return out


# --------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    f64 = torch.float64
    if case["op"] == "rope":
        out, kc, vc = s["out"].to(f64), s["k_cache"].to(f64), s["v_cache"].to(f64)
        rot = case["rot"]
        turn = torch.polar(torch.full_like(s["freq"], s["factor"], dtype=f64),
                           torch.zeros_like(s["freq"], dtype=f64))
        phase = torch.outer(s["pos"].to(f64), s["freq"].to(f64))
        spin = (turn * torch.exp(1j * phase))[:, None, :]          # a complex number per token and pair

        def rotate(x):
            y = x.to(f64).clone()
            if case["interleaved"]:
                y[..., :rot] = torch.view_as_real(
                    torch.view_as_complex(y[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * spin).flatten(-2)
            else:
                z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * spin
                y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
            return y

        keep = s["slots"] >= 0
        where = s["slots"][keep]
        out[keep] = rotate(s["q"])[keep]
        kc.view(-1, case["hkv"], case["d"])[where] = rotate(s["k"])[keep]
        vc.view(-1, case["hkv"], case["d"])[where] = s["v"].to(f64)[keep]
        return out, kc, vc
    hq, hkv = case["hq"], case["hkv"]
    lens, starts = s["lens_host"], s["starts_host"]
    chunks = s["chunks"] if case["op"] == "prefill" else [1] * len(lens)
    if sum(c * n for c, n in zip(chunks, lens)) * hq * case["d"] > 4e12:
        return None
    result = torch.zeros(s["q"].shape, dtype=f64, device=s["q"].device)
    first = 0
    for i, (c, n) in enumerate(zip(chunks, lens)):
        for h in range(hq) if n else ():
            tokens = torch.arange(n, device=s["q"].device)
            block = s["table"][i].long()[tokens // BS]
            k = s["k_cache"][block, tokens % BS, h // (hq // hkv)].to(f64)
            v = s["v_cache"][block, tokens % BS, h // (hq // hkv)].to(f64)
            place = torch.arange(n - c, n, device=s["q"].device)
            away = tokens[None, :] - place[:, None]                  # key position minus query position
            z = s["scale"] * (s["q"][first:first + c, h].to(f64) @ k.T)
            if case["softcap"]:
                z = case["softcap"] * torch.tanh(z / case["softcap"])
            if case["bias"]:
                z = z - float(s["slopes"][h]) * away.abs().to(f64)
            hidden = away > 0
            if case["op"] == "prefill":
                hidden &= tokens[None, :] >= s["prefix_host"][i]
            hidden |= tokens[None, :] < starts[i]
            if case["window"]:
                hidden |= away <= -case["window"]
            z[hidden] = -math.inf
            weight = torch.nan_to_num(torch.softmax(z, dim=-1), nan=0.0)   # a row that sees nothing is zero
            result[first:first + c, h] = weight @ v
        first += c
    return result
