"""The dropout's generator: one block from any counter and key against the three
published vectors of Philox 4x32-10 (Salmon et al. 2011), and the mask's words
against that block, each word in its place (CPU only)."""
import pytest
import torch

import train_ref as ref

LOW = 2 ** 32 - 1


def block(counter, key):
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [b >> 32 ^ c[1] ^ k[0], b & LOW, a >> 32 ^ c[3] ^ k[1], a & LOW]
        k = [k[0] + 0x9E3779B9 & LOW, k[1] + 0xBB67AE85 & LOW]
    return c


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((LOW, LOW, LOW, LOW), (LOW, LOW), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_published_vectors(counter, key, words):
    assert block(counter, key) == list(words)


SEEDS = [(0x299F31D0A4093822, 0x0370734413198A2E), (1 << 32, 1), (1, 1 << 32), (2 ** 64 - 1, 2 ** 63), (7, 0)]


@pytest.mark.parametrize("seed,offset", SEEDS)
def test_words_take_their_places_in_counter_and_key(seed, offset):
    # word n % 4 of the block with counter {n / 4 low, high, offset low, high} and key {seed low, high}
    words = ref.philox_words(4 * 300, seed, offset)
    for i in (0, 1, 2, 77, 299):
        assert words[4 * i:4 * i + 4].tolist() == block((i, 0, offset & LOW, offset >> 32), (seed & LOW, seed >> 32)), i


@pytest.mark.parametrize("seed,offset", SEEDS)
def test_mask_keeps_by_the_words(seed, offset):
    M, H, p = 5, 64, 0.3
    signed = lambda v: v - 2 ** 64 if v >= 2 ** 63 else v  # as the int64 tensor holds it
    keep = ref.mask(M, H, p, torch.tensor([signed(seed), signed(offset)]), "cpu")
    for t, n in ((0, 0), (0, 3), (1, 5), (4, 63)):
        i = t * H + n
        word = block((i // 4, 0, offset & LOW, offset >> 32), (seed & LOW, seed >> 32))[i % 4]
        assert bool(keep[t, n]) == (word >= int(p * 2 ** 32)), (t, n)
