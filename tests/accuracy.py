"""How far results are from 64-bit ones, element by element and as a root mean square."""

# a normal error's rms over N elements lies within a few sqrt(1 / 2N) of its own; at the fewest elements used (about 500)
# 1.15 is five of them
MARGIN = 1.15


def misses(got, want, bound, rms):
    """(elements outside their bound, the error's rms over what it may be): rms holds every element's allowance besides the output's
    rounding, which is taken as it is for these values.  A ratio past MARGIN is a miss."""
    want, bound, rms = (t.to(got.device) for t in (want, bound, rms))
    err = (got.double() - want).abs()
    rounding = want.to(got.dtype).double() - want
    allowed = (rounding.square().mean() + rms.square().mean()).sqrt()
    return int((~(err <= bound)).sum()), (err.square().mean().sqrt() / allowed).item()
