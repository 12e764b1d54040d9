"""Keys and values that make every tile of a long sequence visible in the output: a piece of
it that a join loses, or takes twice, leaves a column off by at least half of itself.

Rows are cut into as many stretches as values have columns; a row's value is 1 in its
stretch's column and 0 elsewhere, so a column of the output is its stretch's share of
the weights, whatever the others are.  Scores come from one positional column alone, with a
course along the sequence that gives each piece a maximum of its own; they are exact in bf16.
The bounds of latent_cases.check_attention are relative to mean, which is the output itself
here (no value is negative): about 1.5 % of a column at 32,768 keys in bf16."""
import numpy as np
import torch

FACTORS = (1.0, 0.5, 2.0, -1.0)  # of the heads' queries, in turn
COURSES = ("equal", "rising", "falling", "peaks")


def scores(course, length):
    """Multiples of 1/16 up to 8."""
    x = np.arange(length) / max(length - 1, 1)
    if course == "equal":
        return np.zeros(length)
    if course == "peaks":
        return np.round(128 * np.abs(np.sin(37 * x) * np.sin(1 + 5 * x))) / 16
    return np.round(128 * (x if course == "rising" else 1 - x)) / 16


def values(length, columns):
    """[length, columns]: row j is 1 in the column of its stretch."""
    v = np.zeros((length, columns))
    v[np.arange(length), np.arange(length) // max(-(-length // columns), 1)] = 1
    return v


def queries(rows, heads, width, column, dtype):
    q = torch.zeros(rows, heads, width)
    q[..., column] = torch.tensor(FACTORS).repeat(-(-heads // 4))[:heads]
    return q.to(dtype)


def mark_cache(cache, table, lens, dc, course):
    """Writes the rows of the sequences into a cache of latent_cases.paged."""
    page = cache.shape[1]
    for n, length in enumerate(lens):
        if length < 1:
            continue
        rows = torch.zeros(length, cache.shape[2])
        rows[:, :dc] = torch.from_numpy(values(length, dc))
        rows[:, dc] = torch.from_numpy(scores(course, length))
        j = np.arange(length)
        cache[torch.from_numpy(table[n][j // page]), torch.from_numpy(j % page)] = rows.to(cache.dtype)
