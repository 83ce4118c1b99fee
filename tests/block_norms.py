"""Relative distances of whole outputs, in units of the type's unit roundoff u.

A value rounded to the type is off by at most u of itself, evenly spread, so
by u / sqrt(3) in the mean square at most; roundings of many values are
independent and keep that as the relative distance of the array, and of a
product with it.  One rounding (a forward output): 0.58 u.  Two (dz, then the
gradient): 0.82 u.  The rest of each bound is for sums in fp32 and for arrays
of few values.  Sums held in the type miss them by far: every rounding of a
running sum adds its own.
"""
ONE_ROUNDING = 0.7
TWO_ROUNDINGS = 1.0


def distance(got, want):
    return float((got.double() - want).norm() / want.norm())
