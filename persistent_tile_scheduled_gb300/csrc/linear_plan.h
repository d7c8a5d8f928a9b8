// How the rows and columns of an epilogue's gradient are dealt out (linear_grad.cu).
// Host-only; each choice comes from the measurement on GB300 quoted beside it.
#pragma once
#include <cstdint>

namespace pts {

constexpr int kGradThreads = 256;   // of a CTA, or twice that
constexpr int kGradMaxCtas = 16;    // CTAs of a cluster: they share an expert's rows

struct GradShape {
    int tx, threads, ctas;   // threads side by side (8 columns each), of a CTA; CTAs that share a block's rows
    int64_t blocks, units;   // of columns; over all experts
};

// room: clusters of kGradMaxCtas that the device holds at once.  So many CTAs are more than
// every device promises to place (8 are), so a cluster has no more than those where it holds
// none, or would take a second wave of them (14 gated: 16384 rows of 512, 16 of them, 28.2
// us, by 8 CTAs 24.8; of 608 31.1 and 26.4).
inline GradShape grad_shape(int64_t rows, int64_t experts, int64_t N, bool gated, bool dbias, int sms, int room)
{
    // Blocks of 64 columns, and as many CTAs of 512 threads (two to an SM; gated, with more
    // registers, one, and two of 256) to one as make a single wave, 8 at most; blocks of 32
    // where columns are few, then also 16 CTAs of 256 threads (us, gelu's tanh form, bf16:
    // 16384 rows of 8192 128 blocks by 2 133, by 4 of 256 threads 134, by 8 142; of 2048 32
    // by 8 38.5, 64 blocks of 32 columns by 4 44; of 1024 32 of 32 by 8 24.5, 16 of 64 by 16
    // 29.7; of 512 16 of 32 by 16 of 256 threads 17.2, by 8 19.1; 9115 gated of 1024 by 256
    // threads 21, by 512 33).  Rows that are no multiple of 32 bytes share those at a
    // block's edges: blocks of 128 columns, unless they are too few for the SMs (9115 rows, by
    // 128 / 64 columns: of 7000 75 / 81, of 5128 69 / 71, of 3848 45 / 51, of 2568, 41 blocks
    // of 64, 37 / 37.5, but of 1928, 31 of them, 31.6 / 27, of 1288 25 / 21).
    // Experts' rows are uneven: where there are many of them a block is shared although a
    // wave is full, so that the largest does not end last (16384 over 8 of 2048, uneven as
    // exp of half a normal / even: 54 / 41, not shared 67 / 37; gated 67 / 68, 76 / 61).
    // Few rows each and more blocks than five waves: wider ones (4000 over 64 of 4096 35 /
    // 20, of 64 columns 32 / 30; gated 44 / 33, 51 / 50).
    const int64_t pieces = N / 8, each = rows / experts, by8 = experts * ((pieces + 7) / 8);
    const bool many = experts > 1, fills = dbias && by8 > sms && by8 <= 2 * sms;   // (a wave without sharing)
    const bool wasteful = many && by8 * 3 <= 2 * sms && by8 * 80 > experts * pieces * 11;   // (more than a tenth of a block)
    int64_t tx = by8 * 8 <= sms || wasteful ? 4 : N % 16 && by8 >= 40 && !fills ? 16 : 8;
    while (tx < 64 && each < 512 && experts * ((pieces + tx - 1) / tx) > 5 * sms) tx *= 2;
    const int64_t blocks = (pieces + tx - 1) / tx, units = experts * blocks;
    int64_t ctas = 1;
    while (units * ctas * 2 <= 2 * sms && each >= 128 * ctas && (ctas < 8 || !dbias)) ctas *= 2;
    while (many && ctas < 8 && units * ctas < 512 && each >= 512 * ctas) ctas *= 2;
    int threads = !gated ? (units <= 2 * sms ? 2 : 1) * kGradThreads
                  : (many && each >= 64 && ((ctas == 1 && units <= 2 * sms) || each >= 512 * ctas)) || (ctas == 1 && units <= sms) ? 2 * kGradThreads : kGradThreads;
    if (dbias && ctas == 8 && units * 16 <= 2 * sms && units <= room && each >= 128 * 8) ctas = kGradMaxCtas, threads = kGradThreads;
    return GradShape{static_cast<int>(tx), threads, static_cast<int>(ctas), blocks, units};
}

}  // namespace pts
