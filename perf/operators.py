"""The paged 4-bit KV cache and the token log probabilities, as measured cases.

Three operators' passes:

  append     the new rows of every sequence: q and k are normalised per head, rotated at their
             positions (one or three axes), and k and v are appended to the paged 4-bit cache;
             the appended rows are then gathered back as the values the cache stands for
             (`kv_append_paged`, `kv_gather_paged`)
  attention  the rows of every sequence attend over its pages (`attention_paged`)
  logprobs   log probability of a given token, entropy and the top alternatives of every row of
             logits (`token_logprobs`)

A cached row is held in blocks of 16 dims: one E4M3 scale s = e4m3(max|y| / 6), and 16 E2M1 codes
e2m1(y / s), both rounded to the nearest, ties to even; a value is code * s. Dim 2i of a row is the
low half of byte i, dim 2i + 1 the high half. Pools: codes [pages, kv heads, page, d / 2] and
scales [pages, kv heads, page, d / 16], for k and for v.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of the dense multi-token-prediction step: latency
        dict(name="append-token", op="append", batch=1, rows=1, ragged=False, q_heads=24,
             kv_heads=4, dim=256, rot=64, axes=1, page=64, ctx=8192),
        # the blocks of eight sequences that accepted different numbers of drafts, far positions
        dict(name="append-blocks", op="append", batch=8, rows=16, ragged=True, q_heads=16,
             kv_heads=8, dim=128, rot=128, axes=1, page=16, ctx=32768),
        # a prompt with image positions (time, height, width)
        dict(name="append-prompt", op="append", batch=1, rows=8192, ragged=False, q_heads=16,
             kv_heads=8, dim=128, rot=128, axes=3, page=128, ctx=77),
        # the tiny drafter's block: the smallest call
        dict(name="attention-tiny", op="attention", batch=1, rows=5, ragged=False, q_heads=4,
             kv_heads=2, dim=64, page=16, ctx=64, causal=False),
        # one token of the dense multi-token-prediction step over 8K keys
        dict(name="attention-token", op="attention", batch=1, rows=1, ragged=False, q_heads=24,
             kv_heads=4, dim=256, page=64, ctx=8192, causal=True),
        # a drafter's block of 16 rows over 4K keys, the rows seeing each other freely
        dict(name="attention-block", op="attention", batch=1, rows=16, ragged=False, q_heads=16,
             kv_heads=8, dim=128, page=64, ctx=4096, causal=False),
        # single tokens of 64 sequences of all lengths up to 8K, odd ones among them
        dict(name="attention-batch", op="attention", batch=64, rows=1, ragged=True, q_heads=16,
             kv_heads=8, dim=128, page=32, ctx=8191, causal=True),
        # eight blocks of 16 drafts to verify over 32K keys each
        dict(name="attention-verify", op="attention", batch=8, rows=16, ragged=False, q_heads=16,
             kv_heads=8, dim=128, page=128, ctx=32768, causal=True),
        # one sampled token's log probability
        dict(name="logprobs-token", op="logprobs", rows=1, vocab=248320, pad=0, top=5,
             dtype="float32", temperature=1.0, masked=False),
        # a block's 16 rows, as the non-greedy round leaves them
        dict(name="logprobs-block", op="logprobs", rows=16, vocab=262144, pad=0, top=8,
             dtype="float32", temperature=0.7, masked=False),
        # rows of an odd vocabulary inside a wider buffer, part of it masked off
        dict(name="logprobs-odd", op="logprobs", rows=37, vocab=4099, pad=13, top=3,
             dtype="float32", temperature=1.3, masked=True),
        # a prompt's tokens scored from 16-bit logits
        dict(name="logprobs-prompt", op="logprobs", rows=1024, vocab=248320, pad=0, top=20,
             dtype="bfloat16", temperature=1.0, masked=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "attention", "attention", "logprobs"))
    if op == "logprobs":
        dtype = rng.choice(("float32", "bfloat16"))
        vocab = _log(rng, 64, 262144)
        most = (1 << 28) // (4 if dtype == "float32" else 2)
        rows = _log(rng, 1, max(1, min(1024, most // vocab)))
        return dict(op=op, rows=rows, vocab=vocab, pad=rng.choice((0, 0, rng.randint(1, 40))),
                    top=rng.randint(0, 20), dtype=dtype,
                    temperature=round(rng.uniform(0.3, 2.0), 2), masked=rng.random() < 0.3)
    dim = rng.choice((64, 128, 128, 256))
    kv = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 2, 3, 4, 6, 8))
    page = rng.choice((16, 32, 64, 128))
    batch = _log(rng, 1, 64)
    if op == "append":
        rows = _log(rng, 1, max(1, (1 << 23) // (batch * kv * dim * max(1, group // 2))))
        rot = rng.choice((dim, dim // 2, dim // 4))
        return dict(op=op, batch=batch, rows=rows, ragged=rng.random() < 0.6, q_heads=kv * group,
                    kv_heads=kv, dim=dim, rot=rot, axes=rng.choice((1, 1, 3)), page=page,
                    ctx=_log(rng, 1, 65536))
    rows = _log(rng, 1, 32)
    most = min(65536, (1 << 28) // (batch * kv * dim), (1 << 33) // (batch * kv * dim * rows * group))
    return dict(op=op, batch=batch, rows=rows, ragged=rng.random() < 0.6, q_heads=kv * group,
                kv_heads=kv, dim=dim, page=page, ctx=_log(rng, 1, most), causal=rng.random() < 0.7)


def _lens(case):
    """Rows already cached and new rows of every sequence (from the case alone)."""
    batch, ctx, rows = case["batch"], case["ctx"], case["rows"]
    if not case["ragged"]:
        return [ctx] * batch, [rows] * batch
    lens = [ctx] + [int(ctx * (b * 0.6180339887 % 1.0)) for b in range(1, batch)]
    return lens, [rows] + [1 + b * 7 % rows for b in range(1, batch)]


def work(case):
    if case["op"] == "logprobs":
        r, v = case["rows"], case["vocab"]
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": r * v * size + r * (12 + 8 * case["top"]), "flops": 6 * r * v}
    lens, new = _lens(case)
    d, kv, q = case["dim"], case["kv_heads"], case["q_heads"]
    row = d // 2 + d // 16
    if case["op"] == "append":
        n = sum(new)
        # q, k, v in, q out; codes and scales written, read back, and the values written
        return {"bytes": n * (4 * d * (2 * q + 2 * kv) + 4 * kv * row + 8 * kv * d),
                "flops": n * d * (10 * (q + kv) + 6 * kv)}
    keys = sum(a + b for a, b in zip(lens, new))
    pairs = sum(b * (a + b) - (b * (b - 1) // 2 if case["causal"] else 0) for a, b in zip(lens, new))
    return {"bytes": keys * kv * 2 * row + 8 * sum(new) * q * d, "flops": 4 * pairs * q * d}


# ------------------------------------------------------------------------------------ inputs
def _quantised(g, pages, kv, page, d):
    """Pools of N(0, 1) rows: codes and scales."""
    y = torch.randn((pages * kv * page, d // 16, 16), generator=g, device=DEV)
    s = (y.abs().amax(-1, keepdim=True) / 6).to(torch.float8_e4m3fn)
    r = (y / s.float()).abs()
    mid = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device=DEV)
    c = torch.bucketize(r, mid, out_int32=True).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)
    c = c.view(pages, kv, page, d // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), s.view(torch.uint8).view(pages, kv, page, d // 16).clone()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["op"] == "logprobs":
        return _prepare_logprobs(case, g)
    lens, new = _lens(case)
    batch, rows, d, kv, q, page = (case[k] for k in ("batch", "rows", "dim", "kv_heads", "q_heads",
                                                     "page"))
    need = [-(-(a + b) // page) for a, b in zip(lens, new)]
    width, pages = max(need), sum(need) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((batch, width), dtype=torch.int32, device=DEV)
    first = 0
    for b, n in enumerate(need):
        table[b, :n] = order[first:first + n]
        first += n
    s = dict(case=case, table=table, seq_len=torch.tensor(lens, dtype=torch.int32, device=DEV),
             n_new=torch.tensor(new, dtype=torch.int32, device=DEV))
    if case["op"] == "attention":
        s["k"], s["ks"] = _quantised(g, pages, kv, page, d)
        s["v"], s["vs"] = _quantised(g, pages, kv, page, d)
        s["q"] = torch.randn((batch, rows, q, d), generator=g, device=DEV)
        s["out"] = torch.zeros((batch, rows, q, d), device=DEV)
    else:
        z = dict(dtype=torch.uint8, device=DEV)
        s["k"], s["v"] = (torch.zeros((pages, kv, page, d // 2), **z) for _ in range(2))
        s["ks"], s["vs"] = (torch.zeros((pages, kv, page, d // 16), **z) for _ in range(2))
        # one projection's output: q | k | v of every row
        s["qkv"] = torch.randn((batch, rows, (q + 2 * kv) * d), generator=g, device=DEV)
        s["q_norm"] = 1 + 0.1 * torch.randn(d, generator=g, device=DEV)
        s["k_norm"] = 1 + 0.1 * torch.randn(d, generator=g, device=DEV)
        half = case["rot"] // 2
        s["inv_freq"] = 1e6 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        pos = s["seq_len"].view(-1, 1) + torch.arange(rows, dtype=torch.int32, device=DEV)
        if case["axes"] == 3:  # time, and a place in a 40-wide picture
            j = torch.arange(rows, dtype=torch.int32, device=DEV).expand(batch, rows)
            start = s["seq_len"].view(-1, 1)
            pos = torch.stack((pos, start + j // 40, start + j % 40))
            s["axis"] = (torch.arange(half, device=DEV) % 3).to(torch.uint8)
            s["pos"] = pos.contiguous()
        else:
            s["axis"], s["pos"] = None, None
        s["q_out"] = torch.zeros((batch, rows, q, d), device=DEV)
        s["k_out"], s["v_out"] = (torch.zeros((batch, kv, rows, d), device=DEV) for _ in range(2))
    if own:
        from speculative_decoding_drafter_dflash_gb300 import binding
        s["cache"] = binding.PagedKv(s["k"], s["ks"], s["v"], s["vs"], s["table"], s["seq_len"])
        if case["op"] == "attention":
            s["ws"] = binding.alloc_workspace(
                binding.attention_paged_workspace_bytes(s["cache"], rows, q))
    return s


def _prepare_logprobs(case, g):
    rows, vocab = case["rows"], case["vocab"]
    x = 2.5 * torch.randn((rows, vocab + case["pad"]), generator=g, device=DEV)
    logits = x.to(getattr(torch, case["dtype"]))[:, :vocab]
    tokens = torch.randint(0, vocab, (rows,), generator=g, device=DEV).to(torch.int32)
    if case["masked"]:  # a grammar that leaves about a third of the vocabulary
        keep = torch.rand((rows, vocab), generator=g, device=DEV) < 0.35
        keep[torch.arange(rows, device=DEV), tokens.long()] = True
        logits.masked_fill_(~keep, -math.inf)
    s = dict(case=case, logits=logits, tokens=tokens)
    s["logprob"], s["entropy"] = (torch.zeros(rows, device=DEV) for _ in range(2))
    s["ids"] = torch.zeros((rows, case["top"]), dtype=torch.int32, device=DEV)
    s["top"] = torch.zeros((rows, case["top"]), device=DEV)
    if own:
        from speculative_decoding_drafter_dflash_gb300 import binding
        s["ws"] = binding.alloc_workspace(
            binding.token_logprobs_workspace_bytes(rows, vocab, case["top"]))
    return s


# ------------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"append": _append, "attention": _attention, "logprobs": _logprobs}[s["case"]["op"]](s)


def _run_own(s):
    from speculative_decoding_drafter_dflash_gb300 import binding
    c = s["case"]
    if c["op"] == "attention":
        binding.attention_paged(s["cache"], s["q"], s["out"], s["ws"], n_new=s["n_new"],
                                causal=c["causal"])
        return s["out"]
    if c["op"] == "append":
        q, k, v = s["qkv"].split((c["q_heads"] * c["dim"], c["kv_heads"] * c["dim"],
                                  c["kv_heads"] * c["dim"]), dim=2)
        binding.kv_append_paged(s["cache"], q, k, v, s["q_out"], n_new=s["n_new"],
                                q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6,
                                inv_freq=s["inv_freq"], positions=s["pos"], axis=s["axis"])
        binding.kv_gather_paged(s["cache"], s["n_new"], s["k_out"], s["v_out"], start=s["seq_len"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    binding.token_logprobs(s["logits"], s["tokens"], s["logprob"], s["entropy"], s["ids"],
                           s["top"], s["ws"], temperature=c["temperature"])
    return {"logprob": s["logprob"], "entropy": s["entropy"], "ids": s["ids"], "top": s["top"]}


def _held(y):
    """What the cache holds for rows y (float64): (codes' values, scales), blocks of 16."""
    y = y.reshape(*y.shape[:-1], -1, 16)
    a = y.abs().amax(-1, keepdim=True) / 6
    e = (torch.frexp(a)[1] - 1).clamp(-6, 8)
    step = torch.ldexp(torch.ones_like(a), e - 3)
    s = (torch.round(a / step) * step).clamp(max=448.0)
    r = torch.where(s > 0, y.abs() / s, torch.zeros_like(y))
    step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0))
    c = (torch.round(r / step) * step).clamp(max=6.0)
    return torch.copysign(c, y), s


def _append(s):
    c = s["case"]
    batch, rows, d, kv, nq, page = (c[k] for k in ("batch", "rows", "dim", "kv_heads", "q_heads",
                                                   "page"))
    x = s["qkv"].view(batch, rows, nq + 2 * kv, d).double()
    q, k, v = x[:, :, :nq], x[:, :, nq:nq + kv], x[:, :, nq + kv:]
    q = q / torch.sqrt((q * q).mean(-1, keepdim=True) + 1e-6) * s["q_norm"].double()
    k = k / torch.sqrt((k * k).mean(-1, keepdim=True) + 1e-6) * s["k_norm"].double()
    i = torch.arange(rows, device=DEV)
    if s["pos"] is None:
        angle = (s["seq_len"].view(-1, 1) + i).double().unsqueeze(-1) * s["inv_freq"]
    else:
        angle = s["pos"].permute(1, 2, 0)[..., s["axis"].long()].double() * s["inv_freq"]
    cos, sin = torch.cos(angle).unsqueeze(2), torch.sin(angle).unsqueeze(2)
    half = c["rot"] // 2

    def turn(y):
        a, b = y[..., :half], y[..., half:2 * half]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, y[..., 2 * half:]), -1)

    q, k = turn(q), turn(k)
    valid = i < s["n_new"].view(-1, 1)
    at = s["seq_len"].view(-1, 1) + i
    b, j = torch.nonzero(valid, as_tuple=True)
    page_id = s["table"][b, (at[b, j] // page)].long()
    slot = (at[b, j] % page).long()
    values = []
    for y, codes, scales in ((k, s["k"], s["ks"]), (v, s["v"], s["vs"])):
        held, scale = _held(y[b, j])
        n = torch.bucketize(held.abs().reshape(-1, kv, d), torch.tensor(E2M1, device=DEV).double())
        n = n.to(torch.uint8) | (torch.signbit(held).reshape(-1, kv, d).to(torch.uint8) << 3)
        n = n.view(-1, kv, d // 2, 2)
        codes[page_id, :, slot] = n[..., 0] | (n[..., 1] << 4)
        scales[page_id, :, slot] = scale.squeeze(-1).to(torch.float8_e4m3fn).view(torch.uint8)
        out = torch.zeros((batch, kv, rows, d), device=DEV)
        out[b, :, j] = (held * scale).reshape(-1, kv, d).float()
        values.append(out)
    q_out = torch.where(valid.view(batch, rows, 1, 1), q, torch.zeros_like(q)).float()
    return {"q": q_out, "k": values[0], "v": values[1]}


def _gathered(codes, scales, table):
    """[B, kv, keys, d] values of every sequence's pages, 32 bits."""
    b, w = table.shape
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)
    c = codes[table.long()]                                    # [B, w, kv, page, d / 2]
    y = torch.stack((lut[(c & 15).int()], lut[(c >> 4).int()]), -1)
    sc = scales[table.long()].view(torch.float8_e4m3fn).float()
    y = y.view(*sc.shape, 16) * sc.unsqueeze(-1)
    return y.flatten(-2).transpose(1, 2).reshape(b, codes.shape[1], -1, 2 * codes.shape[-1])


def _attention(s):
    c = s["case"]
    batch, rows, d, kv, nq = (c[k] for k in ("batch", "rows", "dim", "kv_heads", "q_heads"))
    k = _gathered(s["k"], s["ks"], s["table"])
    q = s["q"].view(batch, rows, kv, nq // kv, d).permute(0, 2, 1, 3, 4).reshape(batch, kv, -1, d)
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    del k
    x = x.view(batch, kv, rows, nq // kv, -1)
    key = torch.arange(x.shape[-1], device=DEV)
    i = torch.arange(rows, device=DEV)
    total = (s["seq_len"] + s["n_new"]).view(-1, 1, 1)
    seen = key < total
    if c["causal"]:
        seen = seen & (key <= s["seq_len"].view(-1, 1, 1) + i.view(1, -1, 1))
    x = x.masked_fill(~seen.view(batch, 1, -1, 1, key.numel()), -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(batch, kv, -1, key.numel()), _gathered(s["v"], s["vs"], s["table"]))
    o = o.view(batch, kv, rows, nq // kv, d).permute(0, 2, 1, 3, 4).reshape(batch, rows, nq, d)
    return torch.where((i < s["n_new"].view(-1, 1)).view(batch, rows, 1, 1), o, s["out"])


def _logprobs(s):
    c = s["case"]
    x = s["logits"].float()
    lowest = x.amax(-1, keepdim=True)
    y = (x - lowest) / c["temperature"]
    e = torch.exp(y)
    total = e.sum(-1, keepdim=True)
    lse = torch.log(total)
    entropy = lse - torch.where(e > 0, e * y, torch.zeros_like(y)).sum(-1, keepdim=True) / total
    lp = y - lse
    logprob = lp.gather(1, s["tokens"].long().unsqueeze(1)).squeeze(1)
    # the order of the values as whole numbers, then the lower index: no two keys are alike
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) << 20
    key = key - torch.arange(c["vocab"], device=DEV)
    ids = torch.topk(key, c["top"], dim=-1).indices
    return {"logprob": logprob, "entropy": entropy.squeeze(1), "ids": ids.to(torch.int32),
            "top": lp.gather(1, ids)}


# ------------------------------------------------------------------------------------ in 64 bits
def _e4m3_values():
    out = [m / 8 * 2.0 ** -6 for m in range(8)]
    out += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.array(out[:-1])                                  # the last pattern is no number


def _nearest(values, x):
    """The nearest of sorted `values` to every x >= 0; a tie goes to the even index."""
    v = torch.tensor(values, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(v, x.contiguous()).clamp(1, len(values) - 1)
    lo = hi - 1
    down, up = x - v[lo], v[hi] - x
    take = torch.where(down == up, hi % 2 == 0, up < down)
    return torch.where(take, v[hi], v[lo])


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention,
            "logprobs": _exact_logprobs}[case["op"]](case, s)


def _exact_append(case, s):
    batch, rows, d, kv, nq, rot = (case[k] for k in ("batch", "rows", "dim", "kv_heads", "q_heads",
                                                     "rot"))
    lens, new = _lens(case)
    out_q = torch.zeros((batch, rows, nq, d), dtype=torch.float64, device=DEV)
    out_k = torch.zeros((batch, kv, rows, d), dtype=torch.float64, device=DEV)
    out_v = torch.zeros_like(out_k)
    freq = s["inv_freq"]
    for b in range(batch):
        n = new[b]
        x = s["qkv"][b, :n].to(torch.float64).view(n, nq + 2 * kv, d)
        if s["pos"] is None:
            p = (lens[b] + torch.arange(n, device=DEV)).to(torch.float64)
            phase = torch.exp(1j * p[:, None] * freq[None, :])
        else:
            p = s["pos"][:, b, :n].to(torch.float64)
            phase = torch.exp(1j * p[torch.arange(rot // 2, device=DEV) % 3].T * freq[None, :])

        def head(z, w):
            z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + 1e-6) * w.to(torch.float64)
            c = torch.complex(z[..., :rot // 2].contiguous(), z[..., rot // 2:rot].contiguous())
            c = c * phase[:, None, :]
            return torch.cat((c.real, c.imag, z[..., rot:]), -1)

        def cached(z):
            t = z.reshape(n, kv, d // 16, 16)
            sc = _nearest(_e4m3_values(), t.abs().max(-1, keepdim=True).values / 6.0)
            c = _nearest(E2M1, t.abs() / torch.where(sc == 0, torch.ones_like(sc), sc))
            return (torch.sign(t) * c * sc).reshape(n, kv, d).transpose(0, 1)

        out_q[b, :n] = head(x[:, :nq], s["q_norm"])
        out_k[b, :, :n] = cached(head(x[:, nq:nq + kv], s["k_norm"]))
        out_v[b, :, :n] = cached(x[:, nq + kv:])
    return {"q": out_q, "k": out_k, "v": out_v}


def _exact_attention(case, s):
    batch, rows, d, kv, nq, page = (case[k] for k in ("batch", "rows", "dim", "kv_heads",
                                                      "q_heads", "page"))
    lens, new = _lens(case)
    out = torch.zeros((batch, rows, nq, d), dtype=torch.float64, device=DEV)
    mag = torch.tensor(E2M1, dtype=torch.float64, device=DEV)

    def values(codes, scales, pages, h):
        c = codes[pages, h].reshape(-1, d // 2).long()
        c = torch.stack((c % 16, c // 16), -1).reshape(-1, d)
        y = mag[c % 8] * (1 - 2 * (c // 8)).to(torch.float64)
        sc = scales[pages, h].reshape(-1, d // 16).view(torch.float8_e4m3fn).to(torch.float64)
        return y * sc.repeat_interleave(16, -1)

    for b in range(batch):
        total = lens[b] + new[b]
        pages = s["table"][b, :-(-total // page)].long()
        last = lens[b] + torch.arange(new[b], device=DEV) if case["causal"] else \
            torch.full((new[b],), total - 1, device=DEV)
        for h in range(kv):
            g = slice(h * (nq // kv), (h + 1) * (nq // kv))
            k = values(s["k"], s["ks"], pages, h)[:total]
            x = torch.einsum("igd,kd->igk", s["q"][b, :new[b], g].to(torch.float64), k) / d ** 0.5
            hide = torch.arange(total, device=DEV)[None, None, :] > last[:, None, None]
            p = torch.softmax(x.masked_fill(hide, -math.inf), -1)
            out[b, :new[b], g] = torch.einsum("igk,kd->igd", p,
                                              values(s["v"], s["vs"], pages, h)[:total])
    return out


def _exact_logprobs(case, s):
    rows = case["rows"]
    logprob, entropy, top = [], [], []
    for first in range(0, rows, 64):
        x = s["logits"][first:first + 64].to(torch.float64)
        lp = torch.log_softmax(x / case["temperature"], -1)
        t = s["tokens"][first:first + 64].long()
        logprob.append(lp[torch.arange(len(t), device=DEV), t])
        p = torch.exp(lp)
        entropy.append(-(p * lp.masked_fill(p == 0, 0.0)).sum(-1))
        top.append(lp.sort(-1, descending=True).values[:, :case["top"]])
    return {"logprob": torch.cat(logprob), "entropy": torch.cat(entropy), "ids": None,
            "top": torch.cat(top)}
