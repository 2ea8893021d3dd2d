"""Plain forms of the prompt and shared-prefix attention, head by head, in 64 and in 32 bits,
and the comparison that the tests of their accuracy share."""
import torch


def causal(n_q, n_k, device="cuda"):
    """[n_q, n_k]: query i sees key j iff j <= i + n_k - n_q."""
    i = torch.arange(n_q, device=device)[:, None] + n_k - n_q
    return torch.arange(n_k, device=device)[None] <= i


def attend(q, k, v, seen, scale, cap=0.0, dtype=torch.float64):
    """softmax(softcap(scale q k^T)) v of one head, rows without a key zero, in dtype (on the
    GPU f32 products are f32: TF32 is off by default)."""
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    z = (q @ k.T) * scale
    if cap:
        z = cap * torch.tanh(z / cap)
    z = z.masked_fill(~seen, -float("inf"))
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m.masked_fill(m == -float("inf"), 0.0))
    l = p.sum(-1, keepdim=True)
    return (p @ v) / l.masked_fill(l == 0, 1.0)


def prompt_forms(q, k, v, cu, ck, scale, cap, dtype):
    """attend() for every sequence and head of a packed call."""
    out = torch.zeros(q.shape, dtype=dtype, device=q.device)
    grp = q.shape[1] // k.shape[1]
    for a, b, c, d in zip(cu, cu[1:], ck, ck[1:]):
        if b > a and d > c:
            seen = causal(b - a, d - c, q.device)
            for h in range(q.shape[1]):
                g = h // grp
                out[a:b, h] = attend(q[a:b, h], k[c:d, g], v[c:d, g], seen, scale, cap, dtype)
    return out


def prefix_forms(q, kp, vp, n_prefix, kc, vc, n_ctx, scale, cap, dtype):
    out = torch.zeros(q.shape, dtype=dtype, device=q.device)
    grp = q.shape[1] // kp.shape[0]
    for b, n in enumerate(n_ctx):
        for h in range(q.shape[1]):
            g = h // grp
            k = torch.cat([kp[g, :n_prefix], kc[b, g, :n]])
            v = torch.cat([vp[g, :n_prefix], vc[b, g, :n]])
            if k.shape[0]:
                seen = torch.ones(1, k.shape[0], dtype=torch.bool, device=q.device)
                out[b, h] = attend(q[b:b + 1, h], k, v, seen, scale, cap, dtype)[0]
    return out


def errors(out, ref):
    """(root mean square, largest) of out - ref."""
    d = (out.double() - ref).flatten()
    return float(d.square().mean().sqrt()), float(d.abs().max())


# The kernels' errors against the plain f32 form's on the same inputs.  On the tensor cores two
# f16 hold a value to 2^-23 at most, and the head_dim / 16 accumulation steps of the large terms
# of a score each cut the sum towards zero, by 2^-24 of it on average (2^-23 at most): 16 u of a
# score at head_dim 256, which a plain f32 sum in blocks holds to some 2 u.  Exponentials (2^-22),
# weights and their sums are f32 on both sides.  So up to eight times, and a low half of an operand
# that is left out, 2^-12 of a value, is a thousand times.
FACTOR = 8.0


def assert_as_good_as_f32(out, plain, ref):
    """out is no further from the 64-bit ref than FACTOR times the plain f32 form, rms and max."""
    assert torch.isfinite(out).all()
    (rms, top), (rms32, top32) = errors(out, ref), errors(plain, ref)
    print(f"rms {rms:.2e} (plain f32 {rms32:.2e}), largest {top:.2e} ({top32:.2e})")
    assert rms <= FACTOR * rms32 and top <= FACTOR * top32, (rms, rms32, top, top32)
