"""Cases and plain forms of the operators around several continuations of one prompt:

  * ``kv``     int8 K/V rows with one fp32 scale each, written into a linear cache or a
               ring and read back (q4g_kv_write_*_i8, q4g_kv_read_*_i8);
  * ``shared`` single-token attention of a batch whose sequences share a prefix, each
               with rows of its own after it (q4g_flash_decode_shared, _i8);
  * ``lp``     log probabilities of given tokens with entropy and the top alternatives
               (q4g_token_logprobs).

Shapes are those of the repository's decoders: full layers with one KV head of 512,
sliding layers with 8 (or 2) KV heads of 256, 16 (or 8) query heads, 262,144 tokens.
"""
from __future__ import annotations

import math

import torch

own = False  # True: the framework's kernels; False: the plain forms


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one decode step of 8 continuations: each appends its row and the rows are read back
        {"name": "kv_step_8", "op": "kv", "form": "slots", "rows": 8, "n_kv": 1, "hd": 512, "capacity": 8192,
         "write": True},
        # sliding layers after a prompt: the ring's newest rows, across its wrap
        {"name": "kv_ring_1531", "op": "kv", "form": "ring", "rows": 1531, "n_kv": 8, "hd": 256, "capacity": 2048,
         "write": True},
        # a full layer's 32K prompt cache handed over from fp16 rows to int8 rows
        {"name": "kv_prompt_32k", "op": "kv", "form": "linear", "rows": 32768, "n_kv": 1, "hd": 512,
         "capacity": 32768, "write": True},
        # rows of a cache gathered in another order (a continuation that leaves the batch)
        {"name": "kv_gather_5003", "op": "kv", "form": "slots", "rows": 5003, "n_kv": 2, "hd": 256,
         "capacity": 32768, "write": False},
        # two drafts after a short prompt: latency
        {"name": "shared_f16_b2_p100", "op": "shared", "i8": False, "batch": 2, "n_q": 16, "n_kv": 1, "hd": 512,
         "prefix": 100, "capacity": 32},
        # eight continuations of a 4K prompt on a full layer
        {"name": "shared_f16_b8_p4096", "op": "shared", "i8": False, "batch": 8, "n_q": 16, "n_kv": 1, "hd": 512,
         "prefix": 4096, "capacity": 512},
        # the same with an int8 cache and a 32K prompt
        {"name": "shared_i8_b8_p32768", "op": "shared", "i8": True, "batch": 8, "n_q": 16, "n_kv": 1, "hd": 512,
         "prefix": 32768, "capacity": 256},
        # many continuations, eight KV heads of 256, a prompt that ends inside a tile
        {"name": "shared_f16_kv8_b24_p1000", "op": "shared", "i8": False, "batch": 24, "n_q": 16, "n_kv": 8, "hd": 256,
         "prefix": 1000, "capacity": 300},
        # the top rung: sixteen continuations of a 128K prompt
        {"name": "shared_f16_b16_p131072", "op": "shared", "i8": False, "batch": 16, "n_q": 16, "n_kv": 1, "hd": 512,
         "prefix": 131072, "capacity": 1024},
        # one decode step's logits with the eight likeliest alternatives
        {"name": "lp_1_top8", "op": "lp", "rows": 1, "vocab": 262144, "top": 8, "temperature": 1.0},
        # a small vocabulary of odd size, sampled at a temperature, no alternatives
        {"name": "lp_300_odd", "op": "lp", "rows": 300, "vocab": 32003, "top": 0, "temperature": 0.7},
        # four scored 64-token chunks with twenty alternatives
        {"name": "lp_256_top20", "op": "lp", "rows": 256, "vocab": 262144, "top": 20, "temperature": 1.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["kv", "shared", "shared", "lp"])
    if op == "kv":
        n_kv, hd = rng.choice([(1, 512), (8, 256), (2, 256)])
        form = rng.choice(["slots", "ring", "linear"])
        rows = max(1, _log(rng, 1, 32768) // n_kv)
        cap = max(rows, _log(rng, 64, 32768))
        return {"op": "kv", "form": form, "rows": rows, "n_kv": n_kv, "hd": hd, "capacity": cap,
                "write": rng.random() < 0.7}
    if op == "shared":
        n_q, n_kv, hd = rng.choice([(16, 1, 512), (16, 8, 256), (8, 1, 512), (8, 2, 256)])
        batch = _log(rng, 1, 64)
        most = min(131072, 16 * 131072 // (batch * n_kv) if batch > 16 else 131072 // n_kv)
        return {"op": "shared", "i8": rng.random() < 0.5, "batch": batch, "n_q": n_q, "n_kv": n_kv, "hd": hd,
                "prefix": _log(rng, 16, max(16, most)), "capacity": _log(rng, 8, 1024)}
    rows = _log(rng, 1, 256)
    return {"op": "lp", "rows": rows, "vocab": _log(rng, 1000, 262144), "top": rng.choice([0, 1, 5, 8, 20, 32]),
            "temperature": rng.choice([1.0, 1.0, 0.7, 1.3])}


# ----------------------------------------------------------------- inputs ----
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, sigma, dtype=torch.float16):
    """N(0, sigma) in `dtype`, made in pieces so that no large fp32 copy is held."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 24
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda", dtype=torch.float32) * sigma
    return out


def _quantized(x):
    """int8 codes and fp32 scales of the rows of fp16 x."""
    codes = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    scales = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    xf, cf, sf = x.reshape(-1, x.shape[-1]), codes.view(-1, x.shape[-1]), scales.view(-1)
    step = 1 << 16
    for i in range(0, xf.shape[0], step):
        c, s = _plain_quantize(xf[i:i + step])
        cf[i:i + step] = c
        sf[i:i + step] = s
    return codes, scales


def _plain_quantize(x):
    xf = x.float()
    # a division by a tensor: by a Python number it may become a product with the reciprocal
    s = xf.abs().amax(dim=-1) / torch.full((), 127.0, dtype=torch.float32, device=x.device)
    safe = torch.where(s > 0, s, torch.ones_like(s))
    c = torch.where(s[..., None] > 0, torch.round(xf / safe[..., None]), torch.zeros_like(xf))
    return c.clamp(-127, 127).to(torch.int8), s


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "kv":
        n, n_kv, hd, cap = case["rows"], case["n_kv"], case["hd"], case["capacity"]
        # keys at the decoder's own scale, values of unit size, rows of differing size
        size = torch.exp(0.5 * torch.randn((n, n_kv, 1), generator=g, device="cuda"))
        if case["write"]:
            st["k"] = (_normal(g, (n, n_kv, hd), hd ** -0.25).float() * size).half()
            st["v"] = (_normal(g, (n, n_kv, hd), 1.0).float() * size).half()
        shape = (n_kv, cap) if case["form"] == "ring" else (cap, n_kv)
        if case["write"]:
            st["cache"] = [torch.zeros(shape + (hd,), dtype=torch.int8, device="cuda"),
                           torch.zeros(shape, dtype=torch.float32, device="cuda"),
                           torch.zeros(shape + (hd,), dtype=torch.int8, device="cuda"),
                           torch.zeros(shape, dtype=torch.float32, device="cuda")]
        else:
            k = _quantized(_normal(g, shape + (hd,), hd ** -0.25))
            v = _quantized(_normal(g, shape + (hd,), 1.0))
            st["cache"] = [k[0], k[1], v[0], v[1]]
        if case["form"] == "slots":
            st["slots"] = torch.randperm(cap, generator=g, device="cuda")[:n].contiguous()
        else:
            room = 3 * cap if case["form"] == "ring" else cap - n
            st["pos0"] = int(torch.randint(0, room + 1, (1,), generator=g, device="cuda").item())
        st["k_out"] = torch.empty((n, n_kv, hd), dtype=torch.float16, device="cuda")
        st["v_out"] = torch.empty((n, n_kv, hd), dtype=torch.float16, device="cuda")
    elif case["op"] == "shared":
        b, n_q, n_kv, hd, p, cap = (case[x] for x in ("batch", "n_q", "n_kv", "hd", "prefix", "capacity"))
        # scores of a standard deviation of about 2
        st["q"] = _normal(g, (b, n_q, hd), 2.0 * hd ** -0.25)
        kv = [_normal(g, (p, n_kv, hd), hd ** -0.25), _normal(g, (p, n_kv, hd), 1.0),
              _normal(g, (b, cap, n_kv, hd), hd ** -0.25), _normal(g, (b, cap, n_kv, hd), 1.0)]
        st["kv"] = [_quantized(x) for x in kv] if case["i8"] else kv
        st["own_len"] = torch.randint(0, cap + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
        st["out"] = torch.empty((b, n_q, hd), dtype=torch.float16, device="cuda")
        if own:
            from int4_q4_gemv_b200 import q4g as Q
            nb = Q.q4g_flash_decode_shared_workspace_bytes(b, n_q, n_kv, hd)
            st["ws"] = torch.empty(nb, dtype=torch.uint8, device="cuda")
    else:
        r, v, n = case["rows"], case["vocab"], case["top"]
        z = _normal(g, (r, v), 3.0, torch.float32)
        st["logits"] = 30.0 * torch.tanh(z / 30.0)  # softcapped, as the decoder's head gives them
        st["targets"] = torch.randint(0, v, (r,), generator=g, device="cuda", dtype=torch.int32)
        st["lp"] = torch.empty(r, dtype=torch.float32, device="cuda")
        st["ent"] = torch.empty(r, dtype=torch.float32, device="cuda")
        st["ids"] = torch.empty((r, n), dtype=torch.int32, device="cuda")
        st["top_lp"] = torch.empty((r, n), dtype=torch.float32, device="cuda")
    return st


# -------------------------------------------------------------------- run ----
def run(state):
    if state["op"] == "kv":
        return _own_kv(state) if own else _plain_kv(state)
    if state["op"] == "shared":
        return _own_shared(state) if own else _plain_shared(state)
    return _own_lp(state) if own else _plain_lp(state)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _own_kv(s):
    from int4_q4_gemv_b200 import q4g as Q
    n, n_kv, hd, cap = s["rows"], s["n_kv"], s["hd"], s["capacity"]
    cache = [t.data_ptr() for t in s["cache"]]
    st = _stream()
    if s["form"] == "ring":
        if s["write"]:
            Q.q4g_kv_write_ring_i8(s["k"].data_ptr(), s["v"].data_ptr(), n, n_kv * hd, n_kv, hd, s["pos0"], cap, *cache,
                                   st)
        Q.q4g_kv_read_ring_i8(*cache, n_kv, hd, s["pos0"], cap, n, s["k_out"].data_ptr(), s["v_out"].data_ptr(),
                              n_kv * hd, st)
    else:
        slots, slot0 = (s["slots"].data_ptr(), 0) if s["form"] == "slots" else (0, s["pos0"])
        if s["write"]:
            Q.q4g_kv_write_linear_i8(s["k"].data_ptr(), s["v"].data_ptr(), n, n_kv * hd, n_kv, hd, slots, slot0, cap,
                                     *cache, st)
        Q.q4g_kv_read_linear_i8(*cache, n_kv, hd, slots, slot0, cap, n, s["k_out"].data_ptr(), s["v_out"].data_ptr(),
                                n_kv * hd, st)
    return s["k_out"], s["v_out"]


def _kv_index(s):
    n, cap = s["rows"], s["capacity"]
    if s["form"] == "slots":
        return s["slots"]
    idx = s["pos0"] + torch.arange(n, device="cuda")
    return idx % cap if s["form"] == "ring" else idx


def _plain_kv(s):
    idx, ring, outs = _kv_index(s), s["form"] == "ring", []
    for i, name in ((0, "k"), (2, "v")):
        codes, scales = s["cache"][i], s["cache"][i + 1]
        if s["write"]:
            c, sc = _plain_quantize(s[name])
            if ring:
                codes[:, idx] = c.transpose(0, 1)
                scales[:, idx] = sc.transpose(0, 1)
            else:
                codes[idx] = c
                scales[idx] = sc
        c = codes[:, idx].transpose(0, 1) if ring else codes[idx]
        sc = scales[:, idx].transpose(0, 1) if ring else scales[idx]
        outs.append((c.float() * sc[..., None]).half().contiguous())
    return tuple(outs)


def _own_shared(s):
    from int4_q4_gemv_b200 import q4g as Q
    dims = (s["batch"], s["n_q"], s["n_kv"], s["hd"])
    tail = (s["out"].data_ptr(), s["ws"].data_ptr(), s["ws"].numel(), _stream())
    if s["i8"]:
        (kc, ks), (vc, vs), (okc, oks), (ovc, ovs) = s["kv"]
        Q.q4g_flash_decode_shared_i8(s["q"].data_ptr(), *dims, kc.data_ptr(), ks.data_ptr(), vc.data_ptr(),
                                     vs.data_ptr(), s["prefix"], okc.data_ptr(), oks.data_ptr(), ovc.data_ptr(),
                                     ovs.data_ptr(), s["capacity"], s["own_len"].data_ptr(), *tail)
    else:
        k, v, ok, ov = s["kv"]
        Q.q4g_flash_decode_shared(s["q"].data_ptr(), *dims, k.data_ptr(), v.data_ptr(), s["prefix"], ok.data_ptr(),
                                  ov.data_ptr(), s["capacity"], s["own_len"].data_ptr(), *tail)
    return s["out"]


def _plain_shared(s):
    b, n_q, n_kv, hd, cap = s["batch"], s["n_q"], s["n_kv"], s["hd"], s["capacity"]
    g = n_q // n_kv
    k, v, ok, ov = [c.float() * sc[..., None] for c, sc in s["kv"]] if s["i8"] else [x.float() for x in s["kv"]]
    q = s["q"].float().view(b, n_kv, g, hd)
    dead = torch.arange(cap, device="cuda")[None, :] >= s["own_len"][:, None]
    out = torch.empty((b, n_kv, g, hd), dtype=torch.float32, device="cuda")
    for h in range(n_kv):
        qh = q[:, h]
        sp = (qh.reshape(b * g, hd) @ k[:, h].t()).view(b, g, -1)
        so = (qh @ ok[:, :, h].transpose(1, 2)).masked_fill(dead[:, None, :], -math.inf)
        sc = torch.cat([sp, so], dim=-1)
        p = torch.exp(sc - sc.amax(dim=-1, keepdim=True))
        del sc
        n = sp.shape[-1]
        acc = (p[..., :n].reshape(b * g, n) @ v[:, h]).view(b, g, hd) + p[..., n:] @ ov[:, :, h]
        out[:, h] = acc / p.sum(dim=-1, keepdim=True)
    return out.view(b, n_q, hd).half()


def _own_lp(s):
    from int4_q4_gemv_b200 import q4g as Q
    n = s["top"]
    Q.q4g_token_logprobs(s["logits"].data_ptr(), s["rows"], s["vocab"], s["vocab"], s["temperature"],
                         s["targets"].data_ptr(), s["lp"].data_ptr(), s["ent"].data_ptr(), n,
                         s["ids"].data_ptr() if n else 0, s["top_lp"].data_ptr() if n else 0, _stream())
    return s["lp"], s["ent"], s["ids"], s["top_lp"]


def _plain_lp(s):
    x, n = s["logits"], s["top"]
    d = (x - x.amax(dim=-1, keepdim=True)) / s["temperature"]
    p = torch.exp(d)
    total = p.sum(dim=-1)
    ln = torch.log(total)
    lp = d.gather(1, s["targets"].long()[:, None])[:, 0] - ln
    ent = ln - (p * d).sum(dim=-1) / total
    if n == 0:
        return lp, ent, s["ids"], s["top_lp"]
    del p
    ids = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :n]
    return lp, ent, ids.to(torch.int32), d.gather(1, ids) - ln[:, None]


# ------------------------------------------------------------------- work ----
def work(case):
    if case["op"] == "kv":
        e = 2 * case["rows"] * case["n_kv"] * case["hd"]  # elements of K and V
        scales = 4 * 2 * case["rows"] * case["n_kv"]
        one = 3 * e + scales  # fp16 rows on one side, codes and scales on the other
        return {"bytes": one * (2 if case["write"] else 1), "flops": 2 * e * (2 if case["write"] else 1)}
    if case["op"] == "shared":
        b, n_q, n_kv, hd, p, cap = (case[x] for x in ("batch", "n_q", "n_kv", "hd", "prefix", "capacity"))
        mean = b * cap // 2  # own rows are between none and all of the capacity
        row = n_kv * ((hd + 4) if case["i8"] else 2 * hd)
        return {"bytes": 2 * (p + mean) * row + 4 * b * n_q * hd, "flops": 4 * n_q * hd * (b * p + mean)}
    r, v, n = case["rows"], case["vocab"], case["top"]
    return {"bytes": 4 * r * v + 12 * r + 8 * r * n, "flops": 5 * r * v}


# ------------------------------------------------------------------ exact ----
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "kv":
        return _exact_kv(s)
    if case["op"] == "shared":
        return _exact_shared(s)
    return _exact_lp(s)


def _exact_kv(s):
    idx, outs = _kv_index(s), []
    for i, name in ((0, "k"), (2, "v")):
        if s["write"]:
            x = s[name].double()
            # the row's scale is an fp32 number, and its code the nearest whole number of scales
            scale = (x.abs().amax(dim=-1) / 127.0).float().double()
            code = torch.where(scale[..., None] > 0, torch.round(x / scale.clamp(min=1e-300)[..., None]),
                               torch.zeros_like(x)).clamp(-127, 127)
        else:
            c, sc = s["cache"][i], s["cache"][i + 1]
            if s["form"] == "ring":
                c, sc = c.transpose(0, 1), sc.transpose(0, 1)
            code, scale = c[idx].double(), sc[idx].double()
        outs.append(code * scale[..., None])
    return tuple(outs)


def _exact_shared(s):
    n_q, n_kv = s["n_q"], s["n_kv"]
    g = n_q // n_kv

    def rows(t, h):
        if s["i8"]:
            return t[0][..., h, :].double() * t[1][..., h].double()[..., None]
        return t[..., h, :].double()

    k, v, ok, ov = s["kv"]
    lens = s["own_len"].tolist()
    out = torch.zeros((s["batch"], n_q, s["hd"]), dtype=torch.float64, device="cuda")
    for h in range(n_kv):
        kp, vp, ko, vo = (rows(t, h) for t in (k, v, ok, ov))
        for b, n in enumerate(lens):
            q = s["q"][b, h * g:(h + 1) * g].double()
            a1, a2 = q @ kp.t(), q @ ko[b, :n].t()
            top = torch.cat([a1, a2], dim=-1).amax(dim=-1, keepdim=True)
            w1, w2 = torch.exp(a1 - top), torch.exp(a2 - top)
            o = w1 @ vp + w2 @ vo[b, :n]
            out[b, h * g:(h + 1) * g] = o / (w1.sum(-1, keepdim=True) + w2.sum(-1, keepdim=True))
    return out


def _exact_lp(s):
    n, lp, ent, ids, tops = s["top"], [], [], [], []
    for r in range(s["rows"]):
        x = s["logits"][r].double() / s["temperature"]
        lse = torch.logsumexp(x, dim=0)
        prob = torch.exp(x - lse)
        lp.append(x[s["targets"][r].long()] - lse)
        ent.append(lse - (prob * x).sum())
        if n:
            order = torch.sort(s["logits"][r], descending=True, stable=True).indices[:n]
            ids.append(order.to(torch.int32))
            tops.append(x[order] - lse)
    if not n:
        return torch.stack(lp), torch.stack(ent), s["ids"], s["top_lp"].double()
    return torch.stack(lp), torch.stack(ent), torch.stack(ids), torch.stack(tops)
