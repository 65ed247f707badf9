"""The bound on a row of q as a sum of two e4m3 terms, over every bf16 number; and
the number of probabilities that the verification adds up before it takes their sum."""
import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def test_two_terms_of_a_bf16_number():
    """y = q 2^-k with the row's largest in (224, 448]: exact from 2^-9 of the largest on, else within 2^-17 of it."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16)
    y = bits.view(torch.bfloat16).float()
    y = y[y <= 448]
    first = y.to(E4M3).float()
    second = (y - first).to(E4M3).float()
    off = (y - first - second).abs().double()
    assert off.max() < 2.0 ** -17 * 224 and off.max() == 2.0 ** -10
    assert off[y >= 2.0 ** -9 * 448].max() == 0 and off[y >= 0.25].max() == 0


def test_words_of_exact_sums():
    """511 values next to 2 stay in the 32 bits of the first word, 512 do not."""
    w = np.nextafter(np.float32(2), np.float32(0))
    per = int((w + np.float32(2)).view(np.uint32)) - 0x40000000
    assert 511 * per < 1 << 32 <= 512 * per
