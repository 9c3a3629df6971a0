"""Plain 64-bit forms of the operators around the layer (residual RMS norm and its quantization, dense
product, balance loss, router gradients), for the tests of their kernels."""
import math

import torch

F64 = torch.float64
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}      # half a step, relative
U = 2.0 ** -24                                                      # one fp32 rounding


def words_to_scales(words, recipe, T):
    """Scale words [K/128, scale_rows] -> fp64 scales [T, K/group]."""
    w = words[:, :T].cpu().contiguous()
    if recipe == 0:
        return w.view(torch.float32).t().to(F64)
    by = w.view(torch.uint8).reshape(w.shape[0], T, 4).transpose(0, 1).reshape(T, -1)
    return torch.exp2(by.to(F64) - 127)


def dequantize(codes, words, recipe):
    T, K = codes.shape
    s = words_to_scales(words, recipe, T)
    q = codes.cpu().view(torch.float8_e4m3fn).float().to(F64)
    return (q.reshape(T, s.shape[1], -1) * s[..., None]).reshape(T, K)


def quantize(x, recipe):
    """bf16 rows -> (codes uint8 [T, K], scale words int32 [K/128, scale_rows]), in the quantizer's fp32 steps."""
    T, K = x.shape
    g = 128 if recipe == 0 else 32
    b = x.float().reshape(T, K // g, g)
    amax = b.abs().amax(-1)
    if recipe == 0:
        s = torch.where(amax > 0, amax * torch.tensor(1.0 / 448.0), torch.ones_like(amax))
        words = s.t().contiguous().view(torch.int32)
    else:
        m, e = torch.frexp(amax)
        e = torch.where(amax > 0, (e - 9 + (m > 0.875).int()).clamp(-127, 127), torch.zeros_like(e))
        s = torch.ldexp(torch.ones_like(amax), e)
        by = (e + 127).to(torch.uint8).reshape(T, K // 128, 4)
        words = by.transpose(0, 1).contiguous().view(torch.int32)[..., 0]
    q = (b / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(T, K)
    out = torch.full((K // 128, (T + 135) // 4 * 4), -1, dtype=torch.int32, device=x.device)   # NaN behind the rows
    out[:, :T] = words
    return q, out


def random_weights(gen, K, N, recipe):
    """(codes, scales) as the transform takes them, and the fp64 matrix [K, N] they stand for."""
    g = 128 if recipe == 0 else 32
    if recipe == 2:
        nib = torch.randint(0, 16, (K, N), generator=gen, dtype=torch.uint8)
        v = torch.tensor(E2M1, dtype=F64)[nib.long()]
        codes = nib[:, 0::2] | (nib[:, 1::2] << 4)
    else:
        codes = torch.randn((K, N), generator=gen).mul(16).to(torch.float8_e4m3fn).view(torch.uint8)
        v = codes.view(torch.float8_e4m3fn).float().to(F64)
    if recipe == 0:
        s = torch.rand((K // g, N), generator=gen) * 0.02 + 0.001
        sv = s.to(F64)
    else:
        s = torch.randint(117, 125, (K // g, N), generator=gen, dtype=torch.uint8)
        sv = torch.exp2(s.to(F64) - 127)
    return codes, s, (v.reshape(K // g, g, N) * sv[:, None]).reshape(K, N)


def act(v, a):
    if a == 1:
        return v.clamp(min=0)
    if a == 2:
        return v * torch.sigmoid(v)
    if a == 3:
        return 0.5 * v * (1 + torch.erf(v / math.sqrt(2)))
    if a == 4:
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def linear(xd, wd, bias, a, res):
    """(y in 64 bits, how far fp32 sums in any order and the activation may be off before the last rounding)."""
    K = wd.shape[0]
    v = xd @ wd
    mag = xd.abs() @ wd.abs()
    if bias is not None:
        v = v + bias.to(F64)
        mag = mag + bias.to(F64).abs()
    # K products added one by one in fp32, a truncation (two half steps) each; the activations'
    # slopes stay under 1.13, their own fp32 steps under 32 roundings of |v|
    off = 1.13 * 2 * K * U * mag + 32 * U * v.abs()
    y = act(v, a)
    if res is not None:
        y = y + res.to(F64)
    return y, off + 2 * U * y.abs()


def token_seq(T, off, mask):
    seq = torch.full((T,), -1, dtype=torch.int64)
    for s in range(len(off) - 1):
        seq[off[s]:off[s + 1]] = s
    return seq if mask is None else torch.where(mask.bool(), seq, torch.full_like(seq, -1))


def probs(l, routing):
    p = torch.sigmoid(l) if routing == 1 else torch.exp(l - l.amax(1, keepdim=True))
    return p / p.sum(1, keepdim=True)


def balance(l, idx, seq, S, k, routing, coef):
    """l fp64 [T, E] -> (loss, counts [S, E], tokens [S + 1], mean [S, E])."""
    E = l.shape[1]
    counts = torch.zeros((S, E), dtype=torch.int32)
    mean, tokens, loss = [], [], l.new_zeros(())
    for s in range(S):
        rows = torch.nonzero(seq == s)[:, 0]
        n = rows.numel()
        tokens.append(n)
        if n == 0:
            mean.append(l.new_zeros(E))
            continue
        counts[s] = torch.bincount(idx[rows].reshape(-1).long(), minlength=E).int()
        mean.append(probs(l[rows], routing).mean(0))
        loss = loss + (counts[s].to(F64) * E / (k * n) * mean[-1]).sum()
    full = sum(n > 0 for n in tokens)
    return coef * loss / max(1, full), counts, torch.tensor(tokens + [full], dtype=torch.int32), torch.stack(mean)


def route_weights(l, idx, routing, renorm, pes, rsf):
    raw = torch.sigmoid(l) if routing == 1 else torch.softmax(l, 1)
    u = raw.gather(1, idx.long())
    if routing == 1 or renorm:
        u = u / u.sum(1, keepdim=True)
    return u * (1.0 if pes is None else pes[idx.long()]) * rsf
