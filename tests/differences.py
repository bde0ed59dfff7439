"""A gradient held to central differences along itself."""


def slope_along(loss, base, grad, step):
    """(slope of ``loss`` at ``base`` along ``grad`` by central differences, <grad, grad>): equal for the gradient of
    ``loss``.  Along a random direction of n elements <grad, v> is |grad| |v| / sqrt(n), lost in any tolerance that is a
    share of |grad| |v|; along itself a gradient of the wrong sign is off by twice, one of another direction and the same
    size by once what is looked at.  ``step``: the change of ``base``, relative to its norm.  (Arrays or tensors in 64 bits.)"""
    size = float((grad * grad).sum())
    eps = step * float((base * base).sum()) ** 0.5 / size ** 0.5
    return (loss(base + eps * grad) - loss(base - eps * grad)) / (2 * eps), size


# The third derivative's part is step^2 times it: with steps of 2^-8 and functions of a few factors (silu, a softmax over
# two logits) under 2^-16 * 64.  fp32 layers: sums of some hundred terms leave y within 2^-18 of its size, which step
# enlarges to 2^-10 |y| |dy| / (|base| |grad|), a ratio of the order of 1 (for w2 <base, grad> = <y, dy>).  Together far
# below 2%, which a gradient has to be wrong by to be told.
STEP, SHARE = 2.0 ** -8, 0.02
