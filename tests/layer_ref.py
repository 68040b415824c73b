"""Plain 64-bit forms of the calls in bcjr_layer.h, on any device, for the tests."""
import torch

BLOCK = 256


def unpack_int4(packed, rows, cols):
    """Codes [rows][cols] of the packed tiles, by the layout in bcjr_layer.h, one place at a time."""
    r = torch.arange(rows, device=packed.device)[:, None]
    c = torch.arange(cols, device=packed.device)[None]
    i, o = c % 128, c % 8
    nibble = o // 2 + 4 * (o % 2)
    byte = 512 * (r % 16 // 8) + 64 * (r % 8) + 16 * (i % 32 // 8) + 4 * (i // 32) + nibble // 2
    return (packed[r // 16, c // 128, byte].long() >> (4 * (nibble % 2))) & 15


def int4_weights(packed, scales, zeros, rows, cols, group):
    q = unpack_int4(packed, rows, cols)
    g = torch.arange(cols, device=packed.device) // (group or cols)
    z = zeros.long()[g].t() if zeros is not None else 8
    return (q - z).double() * scales.double()[g].t()


def quantize(w, group, zero_point, scale_dtype):
    """(codes, scales [groups][rows], zeros or None) from the definition in 64 bits; the scale rounded to its type."""
    rows, cols = w.shape
    group = group or cols
    codes, scales, zeros = torch.empty(rows, cols, dtype=torch.long, device=w.device), [], []
    for c in range(0, cols, group):
        part = w[:, c:c + group].double()
        lo, hi = part.amin(1).clamp(max=0), part.amax(1).clamp(min=0)
        s = ((hi - lo).float() / 15 if zero_point else torch.maximum(hi, -lo).float() / 7).to(scale_dtype)
        d = torch.where(s > 0, s.double(), torch.full_like(s.double(), float("inf")))
        z = torch.round(-lo / d).clamp(0, 15) if zero_point else torch.full_like(lo, 8)
        codes[:, c:c + group] = (torch.round(part / d[:, None]) + z[:, None]).clamp(0, 15).long()
        scales.append(s)
        zeros.append(z)
    return codes, torch.stack(scales), torch.stack(zeros).to(torch.uint8) if zero_point else None


def pack_states(states, L, k):
    """The stream's words by string operations, a sequence at a time."""
    out = []
    for row in states.tolist():
        bits = format(row[0], f"0{L}b") + "".join(format(s % (1 << k), f"0{k}b") for s in row[1:])
        bits += "0" * (-len(bits) % 32)
        out.append([int(bits[i:i + 32], 2) for i in range(0, len(bits), 32)])
    t = torch.tensor(out, dtype=torch.int64)
    return torch.where(t >= 2 ** 31, t - 2 ** 32, t).to(torch.int32)


def random_path(n_seq, n, L, k, seed):
    """States [n_seq][n] (int32) of random paths through the bitshift trellis."""
    gen = torch.Generator().manual_seed(seed)
    s = torch.randint(0, 1 << L, (n_seq,), generator=gen)
    out = [s]
    for _ in range(n - 1):
        s = ((s << k) | torch.randint(0, 1 << k, (n_seq,), generator=gen)) & ((1 << L) - 1)
        out.append(s)
    return torch.stack(out, 1).to(torch.int32)


def hash16(numel, step, seed, device):
    """The 16 random bits of either rounding of every element: (of exp_avg, of exp_avg_sq)."""
    m32 = 0xFFFFFFFF
    h = (torch.arange(numel, device=device) * 0x9E3779B1 + step * 0x632BE5AB + seed * 0x85157AF5) & m32
    h = ((h ^ (h >> 15)) * 0x2C1B3C6D) & m32
    h = ((h ^ (h >> 12)) * 0x297A2D39) & m32
    h = h ^ (h >> 15)
    return h >> 16, h & 0xFFFF


def adamw(p, g, m, v, step, lr, b1, b2, eps, wd, gs=1.0):
    """(p, m, v) after one step, all in 64 bits."""
    g = g.double() * gs
    m = b1 * m.double() + (1 - b1) * g
    v = b2 * v.double() + (1 - b2) * g * g
    p = p.double() * (1 - lr * wd) - lr / (1 - b1 ** step) * m / (v.sqrt() / (1 - b2 ** step) ** 0.5 + eps)
    return p, m, v


def flat_offsets(numels):
    at, out = 0, []
    for n in numels:
        out.append(at)
        at += -(-n // BLOCK) * BLOCK
    return out, at
