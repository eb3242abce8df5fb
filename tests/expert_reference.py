"""Definitions in 64 bits of the operators of the layers under the adapters,
and the bounds that their roundings allow."""
import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def power2(exponent: torch.Tensor) -> torch.Tensor:
    """2 ** exponent in 64 bits, exactly (a device's power may be off by its last bit)."""
    table = torch.tensor([2.0 ** e for e in range(-150, 151)], dtype=torch.float64, device=exponent.device)
    return table[exponent.long() + 150]


def encode(w: torch.Tensor):
    """MXFP4 codes and scale bytes of w (finite values)."""
    v = w.double().view(*w.shape[:-1], w.shape[-1] // 32, 32)
    top = v.abs().amax(-1)
    s = torch.full(top.shape, -127, dtype=torch.long, device=w.device)
    for e in range(-126, 126):
        s = torch.where(top >= 2.0 ** (e + 2), torch.full_like(s, e), s)
    a = v.abs() / power2(s)[..., None]
    best, off = torch.zeros_like(a, dtype=torch.uint8), a.clone()
    for code, value in list(enumerate(E2M1))[1:]:
        away = (a - value).abs()
        better = (away < off) | ((away == off) & (code % 2 == 0))
        best = torch.where(better, torch.full_like(best, code), best)
        off = torch.where(better, away, off)
    code = (best + 8 * torch.signbit(v).to(torch.uint8)).view(w.shape)
    return code[..., 0::2] + 16 * code[..., 1::2], (s + 127).to(torch.uint8)


def decode(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    grid = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=codes.device)
    c = codes.long()
    v = torch.stack((grid[c & 15], grid[c >> 4]), -1).view(*scales.shape, 32)
    f = power2(scales.long() - 127)
    f = torch.where(scales == 255, torch.full_like(f, float("nan")), f)
    return (v * f[..., None]).view(*codes.shape[:-1], codes.shape[-1] * 2)


def forward(x, w, ids, fan):
    """(y, sum of |x| |w|) with zeros in the rows without an expert."""
    y = torch.zeros((len(ids), w.shape[1]), dtype=torch.float64, device=x.device)
    size = torch.zeros_like(y)
    for e in range(w.shape[0]):
        at = (ids == e).nonzero()[:, 0]
        if len(at):
            rows, we = x[at // fan].double(), w[e].double()
            y[at] = rows @ we.T
            size[at] = rows.abs() @ we.abs().T
    return y, size


def backward(dy, x, w, ids, fan):
    """dx, dw and the sums of magnitudes of each."""
    dx = torch.zeros((x.shape[0], x.shape[1]), dtype=torch.float64, device=x.device)
    dw = torch.zeros(w.shape, dtype=torch.float64, device=x.device)
    sx, sw = torch.zeros_like(dx), torch.zeros_like(dw)
    for e in range(w.shape[0]):
        at = (ids == e).nonzero()[:, 0]
        if len(at):
            d, rows, we = dy[at].double(), x[at // fan].double(), w[e].double()
            dx.index_add_(0, at // fan, d @ we)
            sx.index_add_(0, at // fan, d.abs() @ we.abs())
            dw[e] = d.T @ rows
            sw[e] = d.abs().T @ rows.abs()
    return dx, dw, sx, sw


def bound(ref, size, terms):
    """What a bf16 result of `terms` products summed in fp32 may be off: half a step
    of the result (2^-8), and a step of 2^-23 of the sum of magnitudes for every addition
    (tensor cores truncate)."""
    sums = terms * 2.0 ** -23 * size
    return 2.0 ** -8 * (ref.abs() + sums) + sums + 2.0 ** -133


def within(got, ref, limit, what):
    got = got.double()
    bad = ~((got - ref).abs() <= limit)
    assert not bool(bad.any()), "%s: %d of %d values off, the first at %s: %g against %g" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), got[bad][0].item(), ref[bad][0].item())
