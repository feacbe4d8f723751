"""Bounds on whole rows of the attention's results, beside the worst cases of single values (serve_common).

For rows and queries N(0, 1) and softmax scale 1 / sqrt(576), over thousands of keys. A rounding is off by half a step
at most, evenly spread: by 2^-8 / sqrt(3) (bf16) or 2^-11 / sqrt(3) (f16) of a value at most in the mean square.
Roundings are independent, so that their errors add up by their squares.
  out   one rounding of each result and, averaged over thousands of keys, of each probability and value (no more
        than another of each result): a row's error is at most sqrt(2 / 3) 2^-8 of its norm.
  lse   a logit, sum of 576 q k / sqrt(576), has products rounded to f16 at worst: its error is under 2^-11 in
        the mean square, and the lse averages the errors of thousands of logits.
A tile of 128 keys that is lost among 38,000 changes the row by 0.7% and the lse by 0.3%."""
import numpy as np


def check_rows(out, lse, ref_out, ref_lse):
    err = np.linalg.norm(out - ref_out, axis=-1)
    assert (err <= (2 / 3) ** 0.5 * 2.0 ** -8 * np.linalg.norm(ref_out, axis=-1)).all(), "a row's values"
    assert (np.abs(lse - ref_lse) <= 2.0 ** -11).all(), "a row's lse"
