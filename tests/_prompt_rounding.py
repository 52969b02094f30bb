"""How far roundings that are independent of one another take an attention row.

The worst case of a row, every weight off by its half step in the direction that
hurts, grows with the sum of w |v|: over many keys of values with both signs it is
far above what happens, and above what a lost tile of keys would do. Independent
roundings add up as squares do. A weight is off by d w with |d| <= 2^-8 (half a
step of bf16), in the mean of squares at most 2^-16 / 3 (evenly spread over the
half step where it is widest, just above a power of two); a row of D values is off by
the vector sum_j d_j w_j v_j, whose square has the mean

    sum_j 2^-16 / 3 w_j^2 |v_j|^2  (the d_j are independent, in the mean zero),

and the output's own rounding adds 2^-16 / 3 |o|^2 in the same way. Where one key
has nearly all of the weight the square is at most 3 times that (d at its largest);
where many have, their vectors point in D directions and the square is within a
fraction of its mean. So 4 times the mean is not passed (a root mean square of
twice what independent roundings give), and fp32's share is far below it.
"""
import torch


def squares(w, v, o):
    """Mean square of the error vectors [n] of rows with weights w [n, L] (normalised) over values v [L, D] whose exact
    outputs are o [n, D], by independent roundings."""
    return 2.0 ** -16 / 3 * ((w ** 2) @ (v ** 2).sum(1) + (o ** 2).sum(1))


def excess(got, w, v, o):
    """Largest ratio of a row's squared error to 4 times what independent roundings give: at most 1."""
    return float((((got - o) ** 2).sum(1) / (4 * squares(w, v, o)).clamp(min=1e-60)).max())


def weights(q, k, scale, lim):
    """float64 softmax weights [n, L] of queries q [n, D] over keys k [L, D]; row i sees lim[i] keys."""
    x = q.double() @ k.double().T * scale
    see = torch.arange(k.shape[0], device=k.device) < lim[:, None]
    return torch.softmax(x.masked_fill(~see, -float("inf")), 1)


def in_tiles(w, v, tile=128, wrong=None, span=None):
    """The operator as it is computed: weights against a whole-number reference rounded to bf16, tiles of `tile` keys, sums
    in fp32, the output in bf16. `wrong(t)`: the tile of v that tile t's weights meet (None: none)."""
    top = w.amax(1, keepdim=True)
    p = (w / torch.exp2(torch.ceil(torch.log2(top)))).float()
    z, pb = p.double().sum(1, keepdim=True), p.bfloat16().float()
    acc = torch.zeros(w.shape[0], v.shape[1])
    for t in range(-(-w.shape[1] // tile)):
        u = t if wrong is None else wrong(t)
        if u is None:
            continue
        a = pb[:, tile * t:tile * (t + 1)]
        b = v[tile * u:tile * (u + 1)].float()
        m = min(a.shape[1], b.shape[0])
        acc += a[:, :m] @ b[:m]
    return (acc.double() / z).bfloat16().double()
