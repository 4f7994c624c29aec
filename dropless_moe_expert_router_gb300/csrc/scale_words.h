// scale_words.h -- rows of scale bytes read in aligned words.
#pragma once

#include <stdint.h>

namespace moe {

// A row of `n` scale bytes that begins off a word: the bytes before it in its first word, and the words that hold it.
struct ScaleWords {
    int skip, words;
};
constexpr ScaleWords scale_words(uintptr_t row, int n) { return {(int)(row & 3), ((int)(row & 3) + n + 3) / 4}; }

// Whether those words may reach out of the pool, whose first or last word another allocation may share: they begin up to three
// bytes before the row and end up to three behind it, and each of the pool's `lines` rows has one byte at least. Such rows
// are read by their bytes.
constexpr bool scales_at_an_end(long long line, long long lines) { return line < 3 || line >= lines - 3; }

}  // namespace moe
