"""How a bf16 query enters products with e4m3 codes: scaled by a power of two
so that its row's maximum lies in [2^14, 2^15), as the sum of three e5m2 values,
each the rounding of what the ones before left (csrc/tree_attn.cuh,
split_queries).  Every mantissa at every distance from the row's maximum."""
import torch


def _parts(x):
    out = []
    for _ in range(3):
        a = x.to(torch.float8_e5m2).float()
        out.append(a)
        x = x - a
    return out


def test_three_e5m2_values_hold_a_bf16_value():
    mantissa = torch.arange(128, 256, dtype=torch.float64)            # 8 significant bits
    exponent = torch.arange(14, -40, -1, dtype=torch.float64)
    s = (mantissa[None] * 2.0 ** (exponent[:, None] - 7)).float()     # scaled values, exact
    assert torch.equal(s, s.to(torch.bfloat16).float()) and s.max() < 2.0 ** 15
    for sign in (1, -1):
        p = _parts(sign * s)
        assert all(torch.isfinite(x).all() for x in p)
        total = sum(x.double() for x in p)
        err = (total - sign * s.double()).abs()
        assert (err[s >= 2.0 ** -9] == 0).all()
        # the row's maximum is 2^14 at least, so this is 2^-31 of it, and 2^-9 is 2^-23 of it
        assert (err <= 2.0 ** -17).all() and (err == 2.0 ** -17).any()


def test_the_scale_stays_normal():
    """From the largest exponent down to the floor, the scale, its inverse and that times log2(e) / sqrt(128) are
    normal fp32 numbers; the scaled maximum is in range, and below it for smaller rows."""
    tiny = torch.finfo(torch.float32).tiny
    for top in range(0, 255):
        eb = max(top, 23)
        up, down = 2.0 ** (268 - eb - 127), 2.0 ** (eb - 14 - 127)
        assert up * down == 1.0 and tiny <= up < 2.0 ** 128 and down * 1.4426950408889634 / 128 ** 0.5 >= tiny
        top_value = (2 - 2.0 ** -7) * 2.0 ** (max(top, 1) - 127)
        assert top_value * up < 2.0 ** 15 and (top < 23 or top_value * up >= 2.0 ** 14)
