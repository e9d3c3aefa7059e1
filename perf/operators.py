"""Workloads of the speculative-decoding operators on the recurrent state.

Four operators, as a server that drafts tokens uses them one after the other:

  tree     the drafted nodes of a tree read the state (plain, decay-gated or
           delta rule); the state is not changed
  verify   which drafted tokens stand, and the token after them, from the
           target's probabilities and given random numbers: a chain with the
           draft's probabilities, or a tree
  advance  the state moves along the accepted path, each sequence by its own
           number of tokens
  pack     states into a pool of 8-bit slots and back (prefix caching)

``run`` computes an operator in elementary torch operations, or, with ``own``,
by the package's calls. ``exact`` restates each definition in 64 bits, token by
token. Sizes: head size 128 with 16 or 32 heads and 64 sequences is the decode
benchmark of this repository; the others cover its range of head sizes, tree
sizes from one node to 64, vocabularies from a few hundred to 131072.
"""

import math

import numpy as np
import torch

own = False


def _la():
    import causal_linear_attention_la_gb300 as la
    return la


DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one user's chat turn: eight drafted nodes, latency is all that counts
        dict(name="tree one user", op="tree", rule="plain", B=1, H=16, T=8, dk=128, dv=128, dtype="bf16", ragged=False),
        # a busy server: the decode benchmark's 2048 states, sixteen nodes each
        dict(name="tree 2048 states", op="tree", rule="plain", B=64, H=32, T=16, dk=128, dv=128, dtype="bf16", ragged=False),
        # wide trees of different sizes on decay-gated heads
        dict(name="tree wide decay", op="tree", rule="decay", B=48, H=32, T=64, dk=128, dv=128, dtype="bf16", ragged=True),
        # the delta rule, an odd number of nodes
        dict(name="tree delta", op="tree", rule="delta", B=24, H=16, T=27, dk=128, dv=128, dtype="bf16", ragged=True),
        # fp32 inputs, the smaller head
        dict(name="tree f32", op="tree", rule="plain", B=16, H=16, T=13, dk=64, dv=64, dtype="f32", ragged=False),
        # one user's chain of five drafted tokens
        dict(name="chain one user", op="chain", B=1, T=5, V=32000, dtype="f32", ragged=False),
        # a batch of chains over a large vocabulary
        dict(name="chain batch", op="chain", B=64, T=7, V=131072, dtype="f32", ragged=True),
        # trees, bf16 probabilities, a vocabulary that is no multiple of a vector
        dict(name="verify tree", op="verify", B=32, T=31, V=50021, dtype="bf16", accept=3, ragged=True),
        # the 2048 states move by up to six accepted tokens
        dict(name="advance 2048 states", op="advance", rule="plain", B=64, H=32, T=16, most=6, dk=128, dv=128, dtype="bf16"),
        # delta rule, fp32 tokens
        dict(name="advance delta f32", op="advance", rule="delta", B=8, H=16, T=24, most=9, dk=64, dv=64, dtype="f32"),
        # 2048 states leave for the prefix cache
        dict(name="pack 2048 states", op="pack", B=64, H=32, dk=128, dv=128, slots=96),
        # a handful of cached prefixes comes back
        dict(name="unpack few", op="unpack", B=6, H=12, dk=64, dv=64, slots=40),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "chain", "verify", "advance", "pack", "unpack"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("chain", "verify"):
        c = dict(op=op, B=_log(rng, 1, 64), T=_log(rng, 1, 32), V=_log(rng, 300, 131072), dtype=dtype, ragged=rng.random() < 0.5)
        # no dearer than the largest listed case: 64 chains of 8 rows
        while c["B"] * (c["T"] + 1) * c["V"] > 64 * 8 * 131072:
            c["B"] = max(1, c["B"] // 2)
        if op == "verify":
            c["accept"] = rng.randint(0, min(5, c["T"]))
        return c
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 64), (32, 32), (16, 16), (64, 128), (128, 64), (32, 16)])
    c = dict(op=op, B=_log(rng, 1, 64), H=_log(rng, 1, 32), dk=dk, dv=dv)
    if op in ("pack", "unpack"):
        c["slots"] = c["B"] + _log(rng, 1, 40)
        return c
    rule = rng.choice(["plain", "decay", "delta"])
    if op == "tree":
        c.update(rule=rule, T=_log(rng, 1, 64), dtype=dtype, ragged=rng.random() < 0.5)
    else:
        T = _log(rng, 1, 64)
        c.update(rule=rule, T=T, most=rng.randint(1, min(T, 12)), dtype=dtype)
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


def _tokens(g, c, n):
    """q, k, v rows [B,H,n,d] as the tests draw them: N(0,1)/sqrt(d); the delta
    rule's keys have unit norm."""
    B, H, dk, dv = c["B"], c["H"], c["dk"], c["dv"]
    q = torch.randn((B, H, n, dk), generator=g, device="cuda") * dk ** -0.5
    k = torch.randn((B, H, n, dk), generator=g, device="cuda") * dk ** -0.5
    v = torch.randn((B, H, n, dv), generator=g, device="cuda") * dv ** -0.5
    if c["rule"] == "delta":
        k = k / k.norm(dim=-1, keepdim=True)
    return q, k, v


def _state(g, c):
    """A state after 64 tokens of history."""
    rule = c.get("rule", "plain")
    _, k, v = _tokens(g, dict(c, rule=rule), 64)
    f = k if rule == "delta" else torch.where(k >= 0, k + 1, torch.exp(torch.clamp(k, max=0.0)))
    S = torch.einsum("bhni,bhnj->bhij", f, v).contiguous()
    return S, f.sum(2).contiguous()


def _prepare_tree(c, g):
    B, H, T = c["B"], c["H"], c["T"]
    S, z = _state(g, c)
    q, k, v = [x.to(DTYPES[c["dtype"]]).contiguous() for x in _tokens(g, c, T)]
    # a random tree that leans to its latest nodes: parent in [-1, i - 1]
    i = torch.arange(T, device="cuda")
    parent = (torch.rand((B, T), generator=g, device="cuda").sqrt() * (i + 1)).long().clamp(max=T - 1)
    parent = (torch.minimum(parent, i) - 1).to(torch.int32).contiguous()
    s = dict(c=c, S=S, z=z, q=q, k=k, v=v, parent=parent, count=None, alpha=None,
             out=torch.zeros((B, H, T, c["dv"]), dtype=q.dtype, device="cuda"))
    if c["ragged"]:
        s["count"] = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["count"][0] = T
    if c["rule"] == "decay":
        s["alpha"] = 1 - 0.5 * torch.rand((H,), generator=g, device="cuda") ** 2 * 0.5
    return s


def _rows(g, c, rows):
    """Probabilities [B, rows, V]: peaked, as a language model's are."""
    x = torch.randn((c["B"], rows, c["V"]), generator=g, device="cuda").mul_(3.0)
    return x


def _prepare_chain(c, g):
    B, T, V = c["B"], c["T"], c["V"]
    x = _rows(g, c, T + 1)
    draft = torch.softmax(x[:, :T] + 0.6 * torch.randn((B, T, V), generator=g, device="cuda"), -1)
    target = torch.softmax(x, -1).to(DTYPES[c["dtype"]])
    del x
    # tokens drawn from the draft's own distribution
    r = torch.rand((B, T, 1), generator=g, device="cuda", dtype=torch.float64)
    at = torch.cumsum(draft.double(), -1)
    tokens = torch.searchsorted(at, r * at[..., -1:], right=True).clamp(max=V - 1).squeeze(-1).to(torch.int32)
    del at
    s = dict(c=c, target=target.contiguous(), draft=draft.to(DTYPES[c["dtype"]]).contiguous(), tokens=tokens.contiguous(),
             uniform=torch.rand((B, T + 1), generator=g, device="cuda"), count=None)
    if c["ragged"]:
        s["count"] = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    return s


def _prepare_verify(c, g):
    """Trees whose accepted path has c["accept"] nodes: node 0, 1, ... hold the
    tokens that the target's samples give there, the others hang off random
    contexts with tokens of their own."""
    B, T, V, L = c["B"], c["T"], c["V"], c["accept"]
    target = torch.softmax(_rows(g, c, T + 1), -1).to(DTYPES[c["dtype"]]).contiguous()
    uniform = torch.rand((B, T + 1), generator=g, device="cuda")
    i = torch.arange(T, device="cuda")
    parent = (torch.rand((B, T), generator=g, device="cuda") * (i + 1)).long()
    parent = torch.minimum(parent, i) - 1
    parent = torch.where(i < L, i - 1, parent)
    tokens = torch.randint(0, V, (B, T), generator=g, device="cuda")
    if L:
        at = torch.cumsum(target[:, :L].double(), -1)
        hit = torch.searchsorted(at, uniform[:, :L, None].double() * at[..., -1:], right=True).clamp(max=V - 1).squeeze(-1)
        tokens[:, :L] = hit
    s = dict(c=c, target=target, tokens=tokens.to(torch.int32).contiguous(), parent=parent.to(torch.int32).contiguous(),
             uniform=uniform, count=None)
    if c["ragged"]:
        s["count"] = torch.randint(L, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    return s


def _prepare_advance(c, g):
    B, H, T, most = c["B"], c["H"], c["T"], c["most"]
    S, z = _state(g, c)
    _, k, v = [x.to(DTYPES[c["dtype"]]).contiguous() for x in _tokens(g, c, T)]
    n = torch.randint(0, most + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    n[0] = most
    # an increasing choice of nodes, as a path through a tree has them
    path = torch.rand((B, T), generator=g, device="cuda").argsort(-1)[:, :most].sort(-1).values
    path = torch.cat([path, torch.full((B, T - most), -1, device="cuda")], 1)
    path = torch.where(torch.arange(T, device="cuda") < n[:, None], path, -1).to(torch.int32).contiguous()
    s = dict(c=c, S=S, z=z, k=k, v=v, path=path, accepted=n, alpha=None, S_out=torch.zeros_like(S), z_out=torch.zeros_like(z))
    if c["rule"] == "decay":
        s["alpha"] = 1 - 0.5 * torch.rand((H,), generator=g, device="cuda") ** 2 * 0.5
    return s


def _pool(c):
    n, H, dk, dv = c["slots"], c["H"], c["dk"], c["dv"]
    return (torch.zeros((n, H, dk, dv), dtype=torch.uint8, device="cuda"),
            torch.zeros((n, H, dk, dv // min(32, dv)), dtype=torch.uint8, device="cuda"),
            torch.zeros((n, H, dk), device="cuda"))


def _prepare_pack(c, g):
    S, z = _state(g, c)
    codes, scales, z_pool = _pool(c)
    slot = torch.rand((c["slots"],), generator=g, device="cuda").argsort()[:c["B"]].to(torch.int32).contiguous()
    return dict(c=c, S=S, z=z, codes=codes, scales=scales, z_pool=z_pool, slot=slot)


def _prepare_unpack(c, g):
    n, H, dk, dv = c["slots"], c["H"], c["dk"], c["dv"]
    S, z = _state(g, dict(c, B=n))
    codes, scales = _quantise(S)
    slot = torch.randint(0, n, (c["B"],), generator=g, device="cuda", dtype=torch.int32)
    return dict(c=c, codes=codes, scales=scales, z_pool=z, slot=slot,
                S=torch.zeros((c["B"], H, dk, dv), device="cuda"), z=torch.zeros((c["B"], H, dk), device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    make = dict(tree=_prepare_tree, chain=_prepare_chain, verify=_prepare_verify, advance=_prepare_advance,
                pack=_prepare_pack, unpack=_prepare_unpack)[case["op"]]
    return make(case, g)


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------


def _phi(x):
    x = x.float()
    return torch.where(x >= 0, x + 1, torch.exp(torch.clamp(x, max=0.0)))


def _ancestors(parent):
    """[B,T,T] fp32, 1 where node j lies on node i's path (i itself too):
    (I - A)^-1 = sum of the powers of the parent matrix A, by squaring."""
    T = parent.shape[1]
    i = torch.arange(T, device=parent.device)
    a = (parent[:, :, None] == i).float()
    a = a + torch.eye(T, device=parent.device)
    # (I + A)^(2^6) counts walks of up to 64 steps: one to 63 of them are
    # enough for every path, and any positive count says "on the path"
    a = (a @ a > 0).float()
    a = (a @ a > 0).float()
    a = (a @ a > 0).float()
    a = (a @ a > 0).float()
    a = (a @ a > 0).float()
    return (a @ a > 0).float()


def _plain_tree(s):
    S, T = s["S"], s["q"].shape[2]
    anc = _ancestors(s["parent"])[:, None]
    v = s["v"].float()
    if s["c"]["rule"] == "delta":
        q, k = s["q"].float(), s["k"].float()
        below = anc - torch.eye(T, device=S.device)
        m = (k @ k.transpose(-1, -2)) * below + torch.eye(T, device=S.device)
        u = torch.linalg.solve_triangular(m, v - k @ S, upper=False, unitriangular=True)
        o = q @ S + ((q @ k.transpose(-1, -2)) * anc) @ u
    else:
        q, k = _phi(s["q"]), _phi(s["k"])
        w = q @ k.transpose(-1, -2) * anc
        num, den = q @ S, (q * s["z"][:, :, None]).sum(-1, keepdim=True)
        if s["alpha"] is not None:
            depth = anc.sum(-1, keepdim=True)
            a = s["alpha"][None, :, None, None]
            w = w * a ** (depth - depth.transpose(-1, -2)).clamp(min=0)
            num, den = num * a ** depth, den * a ** depth
        o = (num + w @ v) / (den + w.sum(-1, keepdim=True) + EPS)
    o = o.to(s["out"].dtype)
    if s["count"] is not None:
        o = torch.where(torch.arange(T, device=S.device)[None, None, :, None] < s["count"][:, None, None, None], o, s["out"])
    return o


def _sample(w, u):
    """Smallest t with w[0] + ... + w[t] > u * (the sum of w), over the last
    dimension in 64 bits; the last positive entry where rounding leaves none."""
    at = torch.cumsum(w, -1)
    t = torch.searchsorted(at, u[..., None].double() * at[..., -1:], right=True).squeeze(-1)
    last = w.shape[-1] - 1 - torch.flip(w > 0, (-1,)).to(torch.uint8).argmax(-1)
    return torch.where(at[..., -1] > 0, torch.minimum(t, last), -1).to(torch.int32)


def _plain_chain(s):
    p, q, T = s["target"], s["draft"], s["c"]["T"]
    B = p.shape[0]
    b = torch.arange(B, device=p.device)
    x = s["tokens"].long()[..., None]
    px, qx = p[:, :T].gather(-1, x).squeeze(-1).double(), q.gather(-1, x).squeeze(-1).double()
    n_all = s["count"].long() if s["count"] is not None else torch.full((B,), T, device=p.device)
    stands = (s["uniform"][:, :T].double() * qx < px) & (torch.arange(T, device=p.device) < n_all[:, None])
    n = stands.long().cumprod(-1).sum(-1)
    row = p[b, n].double()
    rest = torch.clamp(row - q[b, n.clamp(max=T - 1)].double(), min=0.0)
    use = (n < n_all) & (rest.sum(-1) > 0)
    return n.to(torch.int32), _sample(torch.where(use[:, None], rest, row), s["uniform"][:, T])


def _plain_verify(s):
    p, T = s["target"], s["c"]["T"]
    B = p.shape[0]
    i = torch.arange(T, device=p.device)
    pick = _sample(p.double(), s["uniform"])
    n_all = s["count"].long()[:, None] if s["count"] is not None else T
    parent, tokens = s["parent"].long(), s["tokens"]
    twin = (parent[:, :, None] == parent[:, None]) & (tokens[:, :, None] == tokens[:, None]) & (i[:, None] > i)
    hit = (tokens == pick.gather(1, parent + 1)) & (i < n_all) & ~twin.any(-1)
    on = (_ancestors(s["parent"]) @ (~hit).float()[..., None]).squeeze(-1) == 0
    n = on.sum(-1)
    order = torch.where(on, i, T).sort(-1).values
    path = torch.where(i < n[:, None], order, -1).to(torch.int32)
    last = torch.where(on, i + 1, 0).amax(-1)
    return path, n.to(torch.int32), pick.gather(1, last[:, None]).squeeze(1)


def _plain_advance(s):
    most = s["c"]["most"]
    at = s["path"][:, :most].long().clamp(min=0)[:, None, :, None]
    i = torch.arange(most, device=at.device)
    live = (i < s["accepted"][:, None])[:, None, :, None]
    k = torch.take_along_dim(s["k"], at, 2)
    v = torch.where(live, torch.take_along_dim(s["v"], at, 2).float(), 0.0)
    if s["c"]["rule"] == "delta":
        k = torch.where(live, k.float(), 0.0)
        m = torch.tril(k @ k.transpose(-1, -2), -1) + torch.eye(most, device=k.device)
        u = torch.linalg.solve_triangular(m, v - k @ s["S"], upper=False, unitriangular=True)
        return s["S"] + k.transpose(-1, -2) @ u
    k = torch.where(live, _phi(k), 0.0)
    if s["alpha"] is None:
        return s["S"] + k.transpose(-1, -2) @ v, s["z"] + k.sum(2)
    a = s["alpha"][None, :, None, None]
    n = s["accepted"][:, None, None, None]
    k = k * torch.where(live, a ** (n - 1 - i[:, None]).clamp(min=0), 0.0)
    return s["S"] * a ** n + k.transpose(-1, -2) @ v, s["z"] * (a ** n)[..., 0] + k.sum(2)


def _quantise(S):
    """e4m3 codes and e8m0 scale codes of blocks of min(32, dv) values: the
    scale is the smallest power of two (2^-127 at least) that brings the
    block's largest magnitude to 448 or less."""
    w = min(32, S.shape[-1])
    x = S.unflatten(-1, (-1, w))
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0, e - 9 + (m > 0.875).int(), -127).clamp(min=-127)
    codes = torch.ldexp(x, -e[..., None]).flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (e + 127).to(torch.uint8)


def _plain_pack(s):
    at = s["slot"].long()
    codes, scales = _quantise(s["S"])
    s["codes"].index_copy_(0, at, codes)
    s["scales"].index_copy_(0, at, scales)
    s["z_pool"].index_copy_(0, at, s["z"])
    return s["codes"].view(torch.float8_e4m3fn), s["scales"], s["z_pool"]


def _plain_unpack(s):
    at = s["slot"].long()
    w = min(32, s["c"]["dv"])
    x = s["codes"][at].view(torch.float8_e4m3fn).float().unflatten(-1, (-1, w))
    return torch.ldexp(x, s["scales"][at].int()[..., None] - 127).flatten(-2), s["z_pool"][at]


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------


def run(state):
    s, c = state, state["c"]
    op = c["op"]
    if own:
        la = _la()
        if op == "tree":
            if c["rule"] == "delta":
                return la.decode_tree_delta(s["S"], s["q"], s["k"], s["v"], s["parent"], count=s["count"], out=s["out"])
            return la.decode_tree(s["S"], s["z"], s["q"], s["k"], s["v"], s["parent"], alpha=s["alpha"], eps=EPS,
                                  count=s["count"], out=s["out"])
        if op == "chain":
            return la.verify_chain(s["target"], s["draft"], s["tokens"], s["uniform"], count=s["count"])
        if op == "verify":
            return la.verify_tree(s["target"], s["tokens"], s["parent"], s["uniform"], count=s["count"])
        if op == "advance":
            if c["rule"] == "delta":
                return la.state_advance_delta(s["S"], s["k"], s["v"], s["path"], s["accepted"], S_out=s["S_out"])
            return la.state_advance(s["S"], s["z"], s["k"], s["v"], s["path"], s["accepted"], alpha=s["alpha"],
                                    S_out=s["S_out"], z_out=s["z_out"])
        if op == "pack":
            la.state_pack(s["S"], s["codes"], s["scales"], s["slot"], z=s["z"], z_pool=s["z_pool"])
            return s["codes"].view(torch.float8_e4m3fn), s["scales"], s["z_pool"]
        la.state_unpack(s["codes"], s["scales"], s["slot"], s["S"], z_pool=s["z_pool"], z=s["z"])
        return s["S"], s["z"]
    plain = dict(tree=_plain_tree, chain=_plain_chain, verify=_plain_verify, advance=_plain_advance, pack=_plain_pack,
                 unpack=_plain_unpack)[op]
    return plain(s)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    c, op = case, case["op"]
    B = c["B"]
    if op in ("chain", "verify"):
        T, V, w = c["T"], c["V"], 2 if c["dtype"] == "bf16" else 4
        # a chain: one row of the target and one of the draft, two values a
        # token; a tree: the row of every context on the accepted path
        rows = 2 if op == "chain" else c["accept"] + 1
        return dict(bytes=B * (rows * V * w + T * (2 * w + 12)), flops=2.0 * B * rows * V)
    H, dk, dv = c["H"], c["dk"], c["dv"]
    heads, state = B * H, 4 * dk * dv
    if op in ("pack", "unpack"):
        packed = dk * dv + dk * dv // min(32, dv)
        return dict(bytes=heads * (state + packed + 8 * dk) + 4 * B, flops=3.0 * heads * dk * dv)
    T, w, rule = c["T"], 2 if c["dtype"] == "bf16" else 4, c["rule"]
    z = 0 if rule == "delta" else 4 * dk
    if op == "tree":
        # ragged trees: half the nodes on average
        n = T / 2 if c["ragged"] else T
        rows = n * w * (2 * dk + 2 * dv)
        pairs = n * (n + 1) / 2
        flops = (4 if rule == "delta" else 2) * n * dk * dv + 2 * pairs * (dk + dv) * (2 if rule == "delta" else 1)
        return dict(bytes=heads * (state + z + rows) + 4 * B * T, flops=heads * flops)
    n = c["most"] / 2
    flops = (4 if rule == "delta" else 2) * n * dk * dv
    return dict(bytes=heads * (2 * state + 2 * z + n * w * (dk + dv)) + 4 * B * T, flops=heads * flops)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------


def _phi64(x):
    x = x.double()
    return torch.where(x > 0, x + 1, x.clamp(max=0).exp())


def _exact_tree(s):
    """Every node's own state, from its parent's, one node after the other."""
    c = s["c"]
    out = s["out"].double()
    par = s["parent"].tolist()
    n = s["count"].tolist() if s["count"] is not None else [c["T"]] * c["B"]
    for b in range(c["B"]):
        S, z = {-1: s["S"][b].double()}, {-1: s["z"][b].double()}
        a = s["alpha"].double()[:, None] if s["alpha"] is not None else 1.0
        for i in range(n[b]):
            p = par[b][i]
            v = s["v"][b, :, i].double()
            if c["rule"] == "delta":
                k, q = s["k"][b, :, i].double(), s["q"][b, :, i].double()
                u = v - (k[:, :, None] * S[p]).sum(1)
                S[i] = S[p] + k[:, :, None] * u[:, None]
                out[b, :, i] = (q[:, :, None] * S[i]).sum(1)
            else:
                k, q = _phi64(s["k"][b, :, i]), _phi64(s["q"][b, :, i])
                S[i] = (a[..., None] if torch.is_tensor(a) else a) * S[p] + k[:, :, None] * v[:, None]
                z[i] = a * z[p] + k
                out[b, :, i] = (q[:, :, None] * S[i]).sum(1) / ((q * z[i]).sum(-1, keepdim=True) + EPS)
    return out


def _draw64(w, u):
    w = np.where(w > 0, w, 0.0)
    at = np.cumsum(w)
    if not at[-1] > 0:
        return -1
    above = np.nonzero(at > u * at[-1])[0]
    return int(above[0]) if above.size else int(np.nonzero(w)[0][-1])


def _exact_chain(s):
    c = s["c"]
    tokens, uniform = s["tokens"].cpu().numpy(), s["uniform"].double().cpu().numpy()
    count = s["count"].tolist() if s["count"] is not None else [c["T"]] * c["B"]
    got, nxt = [], []
    for b in range(c["B"]):
        n = 0
        while n < count[b]:
            x = int(tokens[b, n])
            if not uniform[b, n] * float(s["draft"][b, n, x]) < float(s["target"][b, n, x]):
                break
            n += 1
        w = s["target"][b, n].double().cpu().numpy()
        if n < count[b]:
            rest = np.maximum(w - s["draft"][b, n].double().cpu().numpy(), 0.0)
            w = rest if rest.sum() > 0 else w
        got.append(n)
        nxt.append(_draw64(w, uniform[b, c["T"]]))
    return torch.tensor(got, dtype=torch.int32), torch.tensor(nxt, dtype=torch.int32)


def _exact_verify(s):
    c = s["c"]
    tokens, parent = s["tokens"].tolist(), s["parent"].tolist()
    uniform = s["uniform"].double().cpu().numpy()
    count = s["count"].tolist() if s["count"] is not None else [c["T"]] * c["B"]
    paths, got, nxt = [], [], []
    for b in range(c["B"]):
        at, path = -1, []
        while True:
            x = _draw64(s["target"][b, at + 1].double().cpu().numpy(), uniform[b, at + 1])
            child = [i for i in range(count[b]) if parent[b][i] == at and tokens[b][i] == x]
            if not child:
                break
            at = child[0]
            path.append(at)
        paths.append(path + [-1] * (c["T"] - len(path)))
        got.append(len(path))
        nxt.append(x)
    return tuple(torch.tensor(x, dtype=torch.int32) for x in (paths, got, nxt))


def _exact_advance(s):
    c = s["c"]
    S, z = s["S"].double(), s["z"].double()
    path, n = s["path"].tolist(), s["accepted"].tolist()
    a = s["alpha"].double() if s["alpha"] is not None else torch.ones(c["H"], dtype=torch.float64, device=S.device)
    for b in range(c["B"]):
        for i in path[b][:n[b]]:
            k, v = s["k"][b, :, i].double(), s["v"][b, :, i].double()
            if c["rule"] == "delta":
                u = (S[b] * k[:, :, None]).sum(1)
                S[b] += k[:, :, None] * (v - u)[:, None]
            else:
                f = _phi64(s["k"][b, :, i])
                S[b] = a[:, None, None] * S[b] + f[:, :, None] * v[:, None]
                z[b] = a[:, None] * z[b] + f
    return S if c["rule"] == "delta" else (S, z)


def _e4m3_values():
    """The 128 non-negative codes' values (the last one stands for NaN)."""
    e, m = np.divmod(np.arange(128), 8)
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def _exact_pack(s):
    c = s["c"]
    x = s["S"].double().cpu().numpy()
    w = min(32, c["dv"])
    x = x.reshape(x.shape[:-1] + (-1, w))
    top = np.abs(x).max(-1)
    e = np.where(top > 0, np.ceil(np.log2(np.maximum(top, 1e-300) / 448.0)), -127.0).clip(-127, None)
    e = np.where((top > 0) & (top <= 448.0 * 2.0 ** (e - 1)) & (e > -127), e - 1, e)
    y = np.abs(x) * 2.0 ** -e[..., None]
    # steps of the format around each value, ties to the even code
    step = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
    y = np.sign(x) * np.round(y / step) * step
    codes = np.zeros((c["slots"], c["H"], c["dk"], c["dv"]))
    scales = np.zeros((c["slots"], c["H"], c["dk"], c["dv"] // w), np.uint8)
    z = np.zeros((c["slots"], c["H"], c["dk"]))
    at = s["slot"].tolist()
    codes[at] = y.reshape(s["S"].shape)
    scales[at] = (e + 127).astype(np.uint8)
    z[at] = s["z"].double().cpu().numpy()
    return torch.from_numpy(codes), torch.from_numpy(scales), torch.from_numpy(z)


def _exact_unpack(s):
    c = s["c"]
    at = s["slot"].tolist()
    code = s["codes"].cpu().numpy()[at]
    x = np.where(code >= 128, -1.0, 1.0) * _e4m3_values()[code & 127]
    e = s["scales"].cpu().numpy()[at].astype(np.float64) - 127
    x = x * np.repeat(2.0 ** e, min(32, c["dv"]), axis=-1)
    return torch.from_numpy(x), s["z_pool"].double()[at]


def exact(case, seed):
    s = prepare(case, seed)
    return dict(tree=_exact_tree, chain=_exact_chain, verify=_exact_verify, advance=_exact_advance, pack=_exact_pack,
                unpack=_exact_unpack)[case["op"]](s)
